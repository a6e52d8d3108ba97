// Gated feed-forward block on NVFP4 operands: one product gives the gate's
// and the up projection's pre-activations of a token and column to the same
// lane, and the activation, the product of the two and the cast to the output
// type happen there, so neither pre-activation goes to memory.
//
//   [a | u] = deq(X) . deq(W)^T,  X [M][K], W [2F][K] (F gate rows, F up rows)
//   forward:   h  = act(a) u                                   [M][F]
//   gradient:  da = dh u act'(a),  du = dh act(a)              [M][da F | du F]
//
// with a and u recomputed from the quantized operands (4 M F K flops again;
// keeping them would cost 8 M F bytes of HBM traffic and memory).
#include "gemm_device.hpp"

namespace nvfp4 {

// ---- the activations ------------------------------------------------------
// SiLU a sigma(a) and the tanh form of GELU, a sigma(2z) with z = c (a +
// 0.044715 a^3), c = sqrt(2 / pi) (since (1 + tanh z) / 2 = sigma(2z), which
// keeps the relative precision of small values).  sigma(y) and 1 - sigma(y)
// both come from t = e^-|y| <= 1, so neither overflows nor cancels.
constexpr int kSilu = 0, kGelu = 1;
constexpr float kGeluC2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)

struct Sigmoid { float s, om; };  // sigma(y), 1 - sigma(y)

__device__ __forceinline__ Sigmoid sigmoid(float y) {
  const float t = __expf(-fabsf(y));
  const float r = __builtin_amdgcn_rcpf(1.0f + t);
  return y >= 0.0f ? Sigmoid{r, t * r} : Sigmoid{t * r, r};
}

template <int ACT>
__device__ __forceinline__ float act_value(float a) {
  if (ACT == kSilu) return a * sigmoid(a).s;
  return a * sigmoid(kGeluC2 * __builtin_fmaf(0.044715f * a * a, a, a)).s;
}

// act(a) and act'(a)
template <int ACT>
__device__ __forceinline__ void act_both(float a, float& h, float& slope) {
  if (ACT == kSilu) {
    const Sigmoid g = sigmoid(a);
    h = a * g.s;
    slope = __builtin_fmaf(h, g.om, g.s);
  } else {
    const Sigmoid g = sigmoid(kGeluC2 * __builtin_fmaf(0.044715f * a * a, a, a));
    h = a * g.s;
    // past |a| = 16 sigma is 0 or 1 in fp32 and the second term vanishes; the
    // clamp keeps its factors finite there
    const float b = fminf(fmaxf(a, -16.0f), 16.0f);
    slope = __builtin_fmaf(b * g.s * g.om, kGeluC2 * __builtin_fmaf(0.134145f * b, b, 1.0f), g.s);
  }
}

// stores one value and returns the magnitude stored
__device__ __forceinline__ float put(const FfnArgs& p, int64_t idx, float v) {
  if (p.bf16) {
    const uint32_t h = bf16_rne(v);
    static_cast<uint16_t*>(p.out)[idx] = (uint16_t)h;
    return fabsf(__uint_as_float(h << 16));
  }
  static_cast<float*>(p.out)[idx] = v;
  return fabsf(v);
}

__device__ __forceinline__ float get(const FfnArgs& p, int64_t idx) {
  return p.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p.dh)[idx] << 16)
                : static_cast<const float*>(p.dh)[idx];
}

// one element (m, n) of the block from its two pre-activations
template <int ACT, bool GRAD>
__device__ __forceinline__ void emit(const FfnArgs& p, int64_t m, int64_t n, float a, float u, float& amax) {
  if (GRAD) {
    float h, slope;
    act_both<ACT>(a, h, slope);
    const float d = get(p, m * p.F + n);
    amax = fmaxf(amax, put(p, m * 2 * p.F + n, d * u * slope));
    amax = fmaxf(amax, put(p, (m * 2 + 1) * p.F + n, d * h));
  } else {
    put(p, m * p.F + n, act_value<ACT>(a) * u);
  }
}

// ---- any shape ------------------------------------------------------------
// A tile of 128 rows x 64 columns takes 64 gate and 64 up rows of W: wave wn's
// 64 rows of the 128-row B tile are 32 gate rows, then the up rows of the same
// columns, so the accumulators of MFMA tile-columns j and j + 2 of a wave are
// the two pre-activations of the same elements.
template <int BN>
struct PairedRows {
  int64_t n0, F;
  __device__ __forceinline__ int64_t operator()(int r) const {
    const int half = r % (BN / 2), up = half / (BN / 4);
    return min(n0 + (r / (BN / 2)) * (BN / 4) + half % (BN / 4), F - 1) + up * F;
  }
};

template <bool GRAD, bool ALIGNED>
__global__ __launch_bounds__(kGemmThreads, 1) void k_ffn(FfnArgs p) {
  constexpr int BM = 128, BN = 128, TI = BM / 32, TJ = BN / 32;
  __shared__ GemmStage<BM, BN> smem[2];
  const int64_t m0 = (int64_t)blockIdx.y * BM, n0 = (int64_t)blockIdx.x * (BN / 2);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int li = lane & 15, lg = lane >> 4;

  floatx4 acc[TI][TJ];
  general_tile<BM, BN, ALIGNED>(p.g, m0, PairedRows<BN>{n0, p.F}, smem, acc, wm, wn, li, lg);

  const float inv_a = __fdiv_rn(1.0f, p.g.a_ts[0]), inv_b = __fdiv_rn(1.0f, p.g.b_ts[0]);
  const int64_t mrow = m0 + wm * (BM / 2) + lg * 4, ncol = n0 + wn * (BN / 4) + li;
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
#pragma unroll
    for (int j = 0; j < TJ / 2; ++j) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t m = mrow + i * 16 + r, n = ncol + j * 16;
        if (m >= p.g.M || n >= p.F) continue;
        const float a = (acc[i][j][r] * inv_a) * inv_b, u = (acc[i][j + TJ / 2][r] * inv_a) * inv_b;
        if (p.act == kSilu)
          emit<kSilu, GRAD>(p, m, n, a, u, amax);
        else
          emit<kGelu, GRAD>(p, m, n, a, u, amax);
      }
    }
  }
  if (GRAD && p.g.amax) amax_to(p.g, amax);
}

template <bool GRAD>
static void launch_ffn_t(const FfnArgs& p, int, hipStream_t st) {
  const GemmArgs& g = p.g;
  const bool aligned = g.K % kBK == 0 && ((uintptr_t)g.a_codes % 16 == 0) && ((uintptr_t)g.b_codes % 16 == 0) &&
                       ((uintptr_t)g.a_scales % 8 == 0) && ((uintptr_t)g.b_scales % 8 == 0);
  const dim3 grid((unsigned)((p.F + 63) / 64), (unsigned)((g.M + 127) / 128));
  if (aligned)
    hipLaunchKernelGGL((k_ffn<GRAD, true>), grid, dim3(kGemmThreads), 0, st, p);
  else
    hipLaunchKernelGGL((k_ffn<GRAD, false>), grid, dim3(kGemmThreads), 0, st, p);
}

void launch_ffn(const FfnArgs& p, int cus, hipStream_t st) {
  if (p.g.amax) launch_zero_amax(p.g.amax, st);
  if (p.dh)
    launch_ffn_t<true>(p, cus, st);
  else
    launch_ffn_t<false>(p, cus, st);
}

}  // namespace nvfp4
