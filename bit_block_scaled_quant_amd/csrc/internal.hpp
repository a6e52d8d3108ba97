// Launchers shared by the C-ABI entry points (host side of the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace nvfp4 {

struct QuantArgs {
  const void* x;
  bool bf16;
  int64_t rows, cols;
  int rounding;  // 0 RNE, 1 SR
  uint64_t seed;
  bool rht;
  uint32_t rht_mask;
  bool two_d;
  uint8_t* codes;
  uint8_t* scales;
  float* tensor_scale;
  uint8_t* codes_t;  // may be null
  uint8_t* scales_t;
  bool amax_given;   // tensor_scale[1] already holds the amax: skip pass 1
};

void launch_quantize(const QuantArgs& a, int cus, hipStream_t st);

// x [rows][cols] quantized rowwise (no transform) and columnwise (the rows
// of x^T, with the transform when rht_t) in one pair of passes
struct CastTransposeArgs {
  const void* x;
  bool bf16;
  int64_t rows, cols;
  int rounding;  // 0 RNE, 1 SR (both copies)
  uint64_t seed, seed_t;
  bool rht_t;
  uint32_t rht_mask;
  uint8_t* codes;
  uint8_t* scales;
  float* tensor_scale;
  uint8_t* codes_t;
  uint8_t* scales_t;
  float* tensor_scale_t;  // may equal tensor_scale when rht_t is off
  uint32_t stream_t;      // SR stream of the columnwise copy: 0, or 1 for nvfp4_quantize's copy
  bool amax_given;        // tensor_scale[1] already holds the amax (no transform): skip pass 1
};

void launch_cast_transpose(const CastTransposeArgs& a, int cus, hipStream_t st);
void launch_rht(const void* x, bool bf16, int64_t rows, int64_t cols, uint32_t mask, float* y, int cus,
                hipStream_t st);
void launch_dequantize(const uint8_t* codes, const uint8_t* scales, const float* ts, int64_t rows, int64_t cols,
                       bool bf16_out, void* out, int cus, hipStream_t st);

struct GemmArgs {
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const float* a_ts;
  const uint8_t* b_codes;
  const uint8_t* b_scales;
  const float* b_ts;
  int64_t M, N, K;
  float* c;            // fp32 output, or
  uint16_t* c16;       // bf16 output (exactly one of c, c16 is set)
  float beta;          // C = A.B^T + beta * C_old (C_old not read when beta == 0)
  unsigned* amax;      // optional: max |stored C| as float bits (cleared by launch_gemm)
};

void launch_gemm(const GemmArgs& g, int cus, hipStream_t st);
// the same product (beta 0, no amax), K divided among the waves of a workgroup where that is faster
void launch_gemm_split(const GemmArgs& g, int cus, hipStream_t st);
void launch_zero_amax(unsigned* p, hipStream_t st);  // *p = 0 (a kernel: captures into graphs)

// Gated feed-forward block: [a | u] = deq(X) . deq(W)^T with W's first F rows
// the gate's and its last F rows the up projection's
struct FfnArgs {
  GemmArgs g;        // a: X [M][K], b: W [2F][K], N = 2F; g.amax: max |stored gradient|
  int64_t F;
  int act;           // 0 SiLU, 1 GELU (tanh form)
  bool bf16;         // type of dh and out
  const void* dh;    // [M][F]: out = [dh u act'(a) | dh act(a)], [M][2F]; null:
  void* out;         // out = act(a) u, [M][F]
};

void launch_ffn(const FfnArgs& a, int cus, hipStream_t st);

// Distillation from a teacher's top logits
struct DistillArgs {
  const void* logits;  // [T][V], rows `stride` elements apart
  bool bf16;
  int64_t T, V, stride;
  const int32_t* idx;  // [T][K]; entries outside 0 .. V - 1 are absent
  const float* top;    // [T][K]
  int K;
  const float* weight;  // [T] or null (all ones)
  float temperature;
  float* loss;          // [T], or null (gradient alone, from the given lse)
  float* lse;           // [T]
  void* grad;           // [T][V] contiguous, type of the logits, or null (loss alone)
};

constexpr int kDistillMaxK = 1024;

void launch_distill(const DistillArgs& a, int cus, hipStream_t st);

// Embedding lookup and the gradient of its table
struct EmbedArgs {
  const int32_t* tok;  // [T]; outside 0 .. V - 1: a zero row, no gradient
  int64_t T, V, D;
  bool bf16;           // type of table and out, or of dout
  float scale;
  const void* in;      // table [V][D], or dout [T][D]
  void* out;           // [T][D], or the fp32 gradient [V][D]
  // the gradient's workspace:
  uint2* sorted;       // (row, position) in the order of rows, then positions
  uint2* many;         // (first entry, entries) of the rows with many
  uint32_t* count;     // how many those are
};

constexpr int64_t kEmbedMaxTokens = INT64_C(1) << 24;  // of the gradient

void launch_embed(const EmbedArgs& a, int cus, hipStream_t st);
int64_t embed_grad_workspace(int64_t T);  // bytes
void launch_embed_grad(const EmbedArgs& a, void* workspace, int cus, hipStream_t st);

// MXFP4: 32-element blocks of E2M1 codes with E8M0 (power-of-two) scales
struct MxGemmArgs {
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const uint8_t* b_codes;
  const uint8_t* b_scales;
  int64_t M, N, K;
  float* c;
};

void launch_mx_quantize(const void* x, bool bf16, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                        int cus, hipStream_t st);
void launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, bool bf16_out,
                          void* out, int cus, hipStream_t st);
void launch_mx_gemm(const MxGemmArgs& g, hipStream_t st);

}  // namespace nvfp4
