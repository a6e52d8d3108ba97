// Embedding lookup with scaling, and the gradient of its table.
//   out[t]  = scale table[tok_t]                     (a zero row if tok_t is outside 0 .. V - 1)
//   grad[v] = scale sum over {t : tok_t = v} of dout[t]   (fp32, every row written)
#include "internal.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

constexpr int kEmbThreads = 256;

// 16 bytes at any element boundary (rows of an odd length start anywhere)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef int32_t i32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// ---- lookup ---------------------------------------------------------------
// 2^lpr_log2 lanes copy a row, one 16-byte vector each at a time; what is left
// of a row past its last whole vector goes element by element.
template <bool BF16>
__global__ __launch_bounds__(kEmbThreads) void k_embed(EmbedArgs p, int lpr_log2) {
  constexpr int N = BF16 ? 8 : 4, B = BF16 ? 2 : 4;
  const int lpr = 1 << lpr_log2, l = threadIdx.x & (lpr - 1);
  const int64_t rows = (int64_t)gridDim.x * (kEmbThreads >> lpr_log2);
  const int64_t nvec = p.D / N;
  for (int64_t t = ((int64_t)blockIdx.x * kEmbThreads + threadIdx.x) >> lpr_log2; t < p.T; t += rows) {
    const int64_t v = p.tok[t];
    const bool ok = v >= 0 && v < p.V;
    const char* src = static_cast<const char*>(p.in) + (ok ? v : 0) * p.D * B;
    char* dst = static_cast<char*>(p.out) + t * p.D * B;
    for (int64_t i = l; i < nvec; i += lpr) {
      u32x4 o = {0u, 0u, 0u, 0u};
      if (ok) {
        const u32x4 w = *reinterpret_cast<const u32x4_a2*>(src + 16 * i);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          o[k] = BF16 ? bf16_rne(__uint_as_float(w[k] << 16) * p.scale) |
                            (bf16_rne(__uint_as_float(w[k] & 0xFFFF0000u) * p.scale) << 16)
                      : __float_as_uint(__uint_as_float(w[k]) * p.scale);
      }
      *reinterpret_cast<u32x4_a2*>(dst + 16 * i) = o;
    }
    for (int64_t i = nvec * N + l; i < p.D; i += lpr) {
      if (BF16) {
        const uint32_t h = reinterpret_cast<const uint16_t*>(src)[i];
        reinterpret_cast<uint16_t*>(dst)[i] = ok ? (uint16_t)bf16_rne(__uint_as_float(h << 16) * p.scale) : 0;
      } else {
        reinterpret_cast<float*>(dst)[i] = ok ? reinterpret_cast<const float*>(src)[i] * p.scale : 0.0f;
      }
    }
  }
}

// ---- gradient of the table ------------------------------------------------
// A workgroup owns up to 64 consecutive rows of the table and a chunk of
// columns, four columns a lane.  It reads all tokens (they stay in L2) and
// lists those of its rows in the order of their positions, so nothing is
// sorted, counted or scattered beforehand, no two workgroups write one row,
// and every sum has one order.  Rows without tokens are written as zeros.
//
// Tokens are taken kBatch at a time, each wave listing a quarter.  The rows a
// batch names are numbered (their rank in a 64-bit mask) and summed kSlots at
// a time in LDS: group g of 2^lpr_log2 lanes adds every G-th entry to its own
// copy, then the copies are joined in the order of the groups.  A row named
// in a later batch again is read, added to and written.
constexpr int kBatch = 4096, kWaveBatch = kBatch / 4;
constexpr int kSlots = 4;
constexpr int kAhead = 8;  // rows of dout in flight per lane

template <bool BF16>
__device__ __forceinline__ void load4(const EmbedArgs& p, int64_t t, int64_t col, float (&x)[4]) {
  const int64_t i = t * p.D + col;
  if (col + 4 <= p.D) {
    if (BF16) {
      const u32x2_a2 w = *reinterpret_cast<const u32x2_a2*>(static_cast<const uint16_t*>(p.in) + i);
      x[0] = __uint_as_float(w[0] << 16);
      x[1] = __uint_as_float(w[0] & 0xFFFF0000u);
      x[2] = __uint_as_float(w[1] << 16);
      x[3] = __uint_as_float(w[1] & 0xFFFF0000u);
    } else {
      const f32x4_a4 w = *reinterpret_cast<const f32x4_a4*>(static_cast<const float*>(p.in) + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = w[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = 0.0f;
      if (col + k < p.D)
        x[k] = BF16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.in)[i + k] << 16)
                    : static_cast<const float*>(p.in)[i + k];
    }
  }
}

template <bool ADD>
__device__ __forceinline__ void store4(const EmbedArgs& p, int64_t row, int64_t col, f32x4_a4 v) {
  float* dst = static_cast<float*>(p.out) + row * p.D + col;
  if (col + 4 <= p.D) {
    if (ADD) v += *reinterpret_cast<const f32x4_a4*>(dst);
    *reinterpret_cast<f32x4_a4*>(dst) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + k < p.D) dst[k] = ADD ? dst[k] + v[k] : v[k];
  }
}

template <bool BF16>
__global__ __launch_bounds__(kEmbThreads) void k_embed_grad(EmbedArgs p, int lpr_log2, int rows_per, int64_t chunks) {
  __shared__ uint32_t s_list[4][kWaveBatch];  // position in the batch << 6 | row of the workgroup
  __shared__ int s_count[4];
  __shared__ unsigned long long s_mask;
  __shared__ float s_acc[kSlots * kEmbThreads * 4];  // [slot][thread][4]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lpr = 1 << lpr_log2, group = tid >> lpr_log2, groups = kEmbThreads >> lpr_log2;
  const int64_t v0 = (int64_t)(blockIdx.x / chunks) * rows_per;
  const int64_t col = ((int64_t)(blockIdx.x % chunks) * lpr + (tid & (lpr - 1))) * 4;
  const int n = (int)min<int64_t>(rows_per, p.V - v0);
  unsigned long long done = 0;  // rows written so far

  for (int64_t t0 = 0; t0 < p.T; t0 += kBatch) {
    if (tid == 0) s_mask = 0;
    __syncthreads();
    int count = 0;
    unsigned long long mask = 0;
    for (int i = 0; i < kWaveBatch; i += 256) {  // four tokens a lane
      const int64_t t = t0 + wave * kWaveBatch + i + 4 * lane;
      i32x4_a4 tk = {-1, -1, -1, -1};
      if (t + 4 <= p.T) {
        tk = *reinterpret_cast<const i32x4_a4*>(p.tok + t);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (t + k < p.T) tk[k] = p.tok[t + k];
      }
      int found = 0;
      uint32_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t d = (int64_t)tk[k] - v0;
        const bool in = d >= 0 && d < n;
        r[k] = in ? (uint32_t)d : 64u;
        found += in;
      }
      if (__ballot(found > 0) == 0) continue;  // wave-uniform
      int before = found;  // inclusive prefix sum over the lanes
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(before, off);
        if (lane >= off) before += o;
      }
      const int all = __shfl(before, 63);
      int at = count + before - found;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (r[k] < 64u) {
          s_list[wave][at++] = (uint32_t)(wave * kWaveBatch + i + 4 * lane + k) << 6 | r[k];
          mask |= 1ull << r[k];
        }
      }
      count += all;
    }
    if (lane == 0) s_count[wave] = count;
    if (mask) atomicOr(&s_mask, mask);
    __syncthreads();
    const unsigned long long named = s_mask;
    const int c0 = s_count[0], c1 = c0 + s_count[1], c2 = c1 + s_count[2], total = c2 + s_count[3];
    const int nrows = __popcll(named);
    for (int s0 = 0; s0 < nrows; s0 += kSlots) {
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        f32x4_a4 zero = {0.f, 0.f, 0.f, 0.f};
        *reinterpret_cast<f32x4_a4*>(s_acc + (s * kEmbThreads + tid) * 4) = zero;
      }
      if (col < p.D) {
        for (int e0 = group; e0 < total; e0 += kAhead * groups) {
          float x[kAhead][4];
          int slot[kAhead];
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int e = e0 + k * groups;
            slot[k] = kSlots;
            if (e < total) {
              const int w = (e >= c0) + (e >= c1) + (e >= c2);
              const uint32_t it = s_list[w][e - (w == 0 ? 0 : w == 1 ? c0 : w == 2 ? c1 : c2)];
              const int rank = __popcll(named & ((1ull << (it & 63u)) - 1ull)) - s0;
              if (rank >= 0 && rank < kSlots) {
                slot[k] = rank;
                load4<BF16>(p, t0 + (it >> 6), col, x[k]);
              }
            }
          }
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            if (slot[k] < kSlots) {
              float* a = s_acc + (slot[k] * kEmbThreads + tid) * 4;
#pragma unroll
              for (int j = 0; j < 4; ++j) a[j] += x[k][j];
            }
          }
        }
      }
      __syncthreads();
      // join: group g takes slots g, g + groups, ..
      for (int s = group; s < kSlots && s0 + s < nrows; s += groups) {
        unsigned long long m = named;
        for (int i = 0; i < s0 + s; ++i) m &= m - 1;
        const int r = __ffsll(m) - 1;
        f32x4_a4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int g = 0; g < groups; ++g) {
          const float* a = s_acc + (s * kEmbThreads + (g << lpr_log2) + (tid & (lpr - 1))) * 4;
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[j] += a[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] *= p.scale;
        if (col < p.D) {
          if (done >> r & 1)
            store4<true>(p, v0 + r, col, sum);
          else
            store4<false>(p, v0 + r, col, sum);
        }
      }
      __syncthreads();
    }
    done |= named;
  }
  const f32x4_a4 zero = {0.f, 0.f, 0.f, 0.f};
  if (col < p.D)
    for (int r = group; r < n; r += groups)
      if (!(done >> r & 1)) store4<false>(p, v0 + r, col, zero);
}

// ------------------------------------------------------------ launch -----
static int log2_up(int64_t v, int lo, int hi) {
  int l = lo;
  while (l < hi && ((int64_t)1 << l) < v) ++l;
  return l;
}

void launch_embed(const EmbedArgs& a, int cus, hipStream_t st) {
  const int lpr = log2_up(a.D / (a.bf16 ? 8 : 4), 3, 8);
  const int64_t per = kEmbThreads >> lpr, want = (a.T + per - 1) / per;
  const dim3 grid((unsigned)std::min<int64_t>(want, (int64_t)cus * 32));
  if (a.bf16)
    hipLaunchKernelGGL(k_embed<true>, grid, dim3(kEmbThreads), 0, st, a, lpr);
  else
    hipLaunchKernelGGL(k_embed<false>, grid, dim3(kEmbThreads), 0, st, a, lpr);
}

void launch_embed_grad(const EmbedArgs& a, int cus, hipStream_t st) {
  const int lpr = log2_up((a.D + 3) / 4, 4, 8);
  const int64_t chunks = (a.D + ((int64_t)4 << lpr) - 1) / ((int64_t)4 << lpr);
  int rows = 1;  // as many rows a workgroup as leaves 16 workgroups per CU, up to the mask's 64
  while (rows < 64 && (a.V / (2 * rows)) * chunks >= (int64_t)cus * 16) rows *= 2;
  // workgroups past the grid's 2^31 - 1: V * D <= 2^40 keeps the count below 2^40 / (64 * 64)
  const dim3 grid((unsigned)(((a.V + rows - 1) / rows) * chunks));
  if (a.bf16)
    hipLaunchKernelGGL(k_embed_grad<true>, grid, dim3(kEmbThreads), 0, st, a, lpr, rows, chunks);
  else
    hipLaunchKernelGGL(k_embed_grad<false>, grid, dim3(kEmbThreads), 0, st, a, lpr, rows, chunks);
}

}  // namespace nvfp4
