// Distillation from a teacher's top logits.  Row r of the logits (V entries)
// against K entries idx_j, top_j of the teacher:
//   z = logits / tau, q = softmax(z), lse = log sum exp z,
//   p = softmax over the present entries of top / tau,
//   loss_r = w_r sum_j p_j (log p_j - (z_idx_j - lse)),
//   grad_r = (q - sum_j p_j e_idx_j) w_r / tau.
// An entry whose idx lies outside 0 .. V - 1 is absent; a row without entries
// or of weight zero has loss and gradient zero, whatever its logits.
//
// One workgroup per row.  The maximum and the sum of exponentials are taken
// in one pass (each thread keeps its own pair and rescales its sum when its
// maximum grows), then the gradient is written densely and the few entries
// of the teacher are corrected.  All statistics are fp32; every reduction has
// a fixed order, so results repeat bit for bit.
#include "internal.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

constexpr int kDistThreads = 1024;
constexpr int kDistWaves = kDistThreads / 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// rows start at any element, so vectors are only element-aligned
template <bool BF16>
struct Vec16;
template <>
struct Vec16<true> {
  typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
  static constexpr int kN = 8;
};
template <>
struct Vec16<false> {
  typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(4)));
  static constexpr int kN = 4;
};
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <bool BF16>
__device__ __forceinline__ u32x4 dist_load(const char* row, int64_t v) {
  return *reinterpret_cast<const typename Vec16<BF16>::raw*>(row + 16 * v);
}

template <bool BF16>
__device__ __forceinline__ float dist_elem(const u32x4& w, int k) {
  if (!BF16) return __uint_as_float(w[k]);
  return __uint_as_float((k & 1) ? (w[k >> 1] & 0xFFFF0000u) : (w[k >> 1] << 16));
}

template <bool BF16>
__device__ __forceinline__ float dist_at(const char* row, int64_t i) {
  if (!BF16) return reinterpret_cast<const float*>(row)[i];
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
}

template <bool BF16>
__device__ __forceinline__ void dist_put(char* row, int64_t i, float v) {
  if (BF16)
    reinterpret_cast<uint16_t*>(row)[i] = (uint16_t)bf16_rne(v);
  else
    reinterpret_cast<float*>(row)[i] = v;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// a row's maximum m of the logits (before the temperature) and sum of
// exp((x - m) / tau); an empty one is (-inf, 0)
struct MaxSum { float m, s; };

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
  const float m = fmaxf(a.m, b.m), ref = finite_or_zero(m);
  return {m, a.s * exp2_hw((a.m - ref) * c) + b.s * exp2_hw((b.m - ref) * c)};
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}

// N values into a thread's running pair: one rescale for all of them.  The
// difference to the maximum is rounded before it is scaled, so the terms that
// carry the sum (x near m) are the precise ones.
template <int N>
__device__ __forceinline__ void online(MaxSum& t, const float (&x)[N], float c) {
  float m = t.m;
#pragma unroll
  for (int k = 0; k < N; ++k) m = fmaxf(m, x[k]);
  const float ref = finite_or_zero(m);
  float s = t.s * exp2_hw((t.m - ref) * c);
#pragma unroll
  for (int k = 0; k < N; ++k) s += exp2_hw((x[k] - ref) * c);
  t.m = m;
  t.s = s;
}

template <bool BF16, bool LOSS, bool GRAD>
__global__ __launch_bounds__(kDistThreads) void k_distill(DistillArgs p) {
  constexpr int N = Vec16<BF16>::kN;
  __shared__ float s_red[3][kDistWaves];
  __shared__ int32_t s_idx[kDistillMaxK];
  __shared__ float s_p[kDistillMaxK];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x;
  const char* x = static_cast<const char*>(p.logits) + row * p.stride * (BF16 ? 2 : 4);
  const int64_t nvec = p.V / N;
  const float c = kLog2e / p.temperature;

  // the teacher's entry of this thread (K <= kDistThreads)
  const bool mine = tid < p.K;
  int32_t at = -1;
  float t = -INFINITY, z = 0.0f;
  if (mine) {
    at = p.idx[row * p.K + tid];
    if (at < 0 || at >= p.V) at = -1;
    if (at >= 0) {
      t = p.top[row * p.K + tid] / p.temperature;
      z = dist_at<BF16>(x, at);
    }
    s_idx[tid] = at;
  }

  MaxSum st{-INFINITY, 0.0f};
  if (LOSS) {
    for (int64_t v = tid; v < nvec; v += kDistThreads) {
      const u32x4 w = dist_load<BF16>(x, v);
      float e[N];
#pragma unroll
      for (int k = 0; k < N; ++k) e[k] = dist_elem<BF16>(w, k);
      online(st, e, c);
    }
    if (nvec * N + tid < p.V) {
      const float e[1] = {dist_at<BF16>(x, nvec * N + tid)};
      online(st, e, c);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) st = join(st, MaxSum{__shfl_xor(st.m, off), __shfl_xor(st.s, off)}, c);
  }
  const float th = wave_max(t);
  if (lane == 0) {
    s_red[0][wave] = st.m;
    s_red[1][wave] = st.s;
    s_red[2][wave] = th;
  }
  __syncthreads();
  float high = -INFINITY;
  st = MaxSum{-INFINITY, 0.0f};
#pragma unroll
  for (int i = 0; i < kDistWaves; ++i) {
    if (LOSS) st = join(st, MaxSum{s_red[0][i], s_red[1][i]}, c);
    high = fmaxf(high, s_red[2][i]);
  }
  __syncthreads();
  const float e = exp2_hw((t - finite_or_zero(high)) * kLog2e);  // 0 for an absent entry
  const float esum = wave_sum(e);
  if (lane == 0) s_red[0][wave] = esum;
  __syncthreads();
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < kDistWaves; ++i) total += s_red[0][i];
  const bool any = high > -INFINITY;
  const float prob = any ? e / total : 0.0f;
  if (mine) s_p[tid] = prob;
  const float w = !any ? 0.0f : p.weight ? p.weight[row] : 1.0f;

  const bool empty = LOSS ? st.s == 0.0f : p.lse[row] == -INFINITY;  // every logit is -inf
  const float ref = finite_or_zero(st.m);
  const float l2s = empty ? 0.0f : __builtin_amdgcn_logf(st.s);
  if (LOSS) {
    const float lse = empty ? -INFINITY : ref / p.temperature + l2s * kLn2;
    const float logq = empty ? -INFINITY : (z - ref) / p.temperature - l2s * kLn2;
    const float logp = (t - high) - __logf(total);
    const float term = wave_sum(prob > 0.0f && w != 0.0f ? prob * (logp - logq) : 0.0f);
    if (lane == 0) s_red[1][wave] = term;
    __syncthreads();
    if (tid == 0) {
      float l = 0.0f;
      for (int i = 0; i < kDistWaves; ++i) l += s_red[1][i];
      p.loss[row] = w == 0.0f ? 0.0f : l * w;
      p.lse[row] = lse;
    }
  }
  if (!GRAD) return;

  // q of a logit: from the pass above, or from the given lse
  const float lse_in = LOSS || empty ? 0.0f : p.lse[row], inv_tau = 1.0f / p.temperature;
  auto q = [&](float v) {
    return LOSS ? exp2_hw(__builtin_fmaf(v - ref, c, -l2s)) : exp2_hw(__builtin_fmaf(v, inv_tau, -lse_in) * kLog2e);
  };
  const float wt = w / p.temperature;
  char* g = static_cast<char*>(p.grad) + row * p.V * (BF16 ? 2 : 4);
  for (int64_t v = tid; v < nvec; v += kDistThreads) {
    u32x4 o = {0u, 0u, 0u, 0u};
    if (w != 0.0f) {
      const u32x4 d = dist_load<BF16>(x, v);
      float e2[N];
#pragma unroll
      for (int k = 0; k < N; ++k) e2[k] = q(dist_elem<BF16>(d, k)) * wt;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o[k] = BF16 ? bf16_rne(e2[(2 * k) % N]) | (bf16_rne(e2[(2 * k + 1) % N]) << 16) : __float_as_uint(e2[k]);
    }
    *reinterpret_cast<typename Vec16<BF16>::raw*>(g + 16 * v) = o;
  }
  if (nvec * N + tid < p.V)
    dist_put<BF16>(g, nvec * N + tid, w != 0.0f ? q(dist_at<BF16>(x, nvec * N + tid)) * wt : 0.0f);
  __syncthreads();  // the dense gradient is written: correct the teacher's entries
  if (at >= 0 && w != 0.0f) {
    float target = 0.0f;  // an index named twice takes the sum, in the entries' order, from each of its threads
    for (int j = 0; j < p.K; ++j)
      if (s_idx[j] == at) target += s_p[j];
    dist_put<BF16>(g, at, (q(z) - target) * wt);
  }
}

template <bool BF16>
static void launch_distill_t(const DistillArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.T), block(kDistThreads);
  if (!a.grad)
    hipLaunchKernelGGL((k_distill<BF16, true, false>), grid, block, 0, st, a);
  else if (a.loss)
    hipLaunchKernelGGL((k_distill<BF16, true, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((k_distill<BF16, false, true>), grid, block, 0, st, a);
}

void launch_distill(const DistillArgs& a, hipStream_t st) {
  if (a.bf16)
    launch_distill_t<true>(a, st);
  else
    launch_distill_t<false>(a, st);
}

}  // namespace nvfp4
