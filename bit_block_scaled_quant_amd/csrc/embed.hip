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
          o[k] = BF16 ? bf16_pair(__uint_as_float(w[k] << 16) * p.scale, __uint_as_float(w[k] & 0xFFFF0000u) * p.scale)
                      : __float_as_uint(__uint_as_float(w[k]) * p.scale);
      }
      *reinterpret_cast<u32x4_a2*>(dst + 16 * i) = o;
    }
    for (int64_t i = nvec * N + l; i < p.D; i += lpr) {
      if (BF16) {
        const uint32_t h = reinterpret_cast<const uint16_t*>(src)[i];
        reinterpret_cast<uint16_t*>(dst)[i] = ok ? (uint16_t)bf16_pair(__uint_as_float(h << 16) * p.scale, 0.0f) : 0;
      } else {
        reinterpret_cast<float*>(dst)[i] = ok ? reinterpret_cast<const float*>(src)[i] * p.scale : 0.0f;
      }
    }
  }
}

// ---- gradient of the table ------------------------------------------------
// 1. k_embed_fill writes zeros everywhere, which bounds a training batch (2.7
//    GB for [131072][5120]).  The store must wait for nothing and be the only
//    one of its thread: 390 us for one 16-byte store a thread in workgroups of
//    256, 435 for two, 470 for eight, 550 for a grid-stride loop, and 555 when
//    each thread also looks up whether its row has tokens (measured; with that
//    the rows below would not be written twice, 3% of the bytes).
// 2. k_embed_sort: each workgroup sorts 8192 tokens by row, stably, in LDS (24
//    us; as the first workgroups of the fill it is hidden, but the fill then
//    needs the sort's large workgroups and takes 25 us more).  Past 8192 tokens,
//    k_embed_merge merges pairs of sorted runs, each entry finding its place by a
//    binary search, once for each doubling.
// 3. k_embed_sums: the lanes at an entry that begins a row sum the row if it has
//    at most kFew entries; rows with more are summed from a list by workgroups of
//    64 columns.  A lone run's sort leaves the list, so that both kinds go in one
//    launch (76 us, 93 one after the other; 104 with 256 columns, since the
//    longest row then decides); else the lanes of the first kind list those rows
//    for a second launch.
// Every sum has one order: that of the positions, cut into equal parts for the
// groups that share a row.
//
// One launch in which every workgroup owned 64 rows, read all tokens and
// listed its own took 538 us for 8192 tokens of [131072][5120], since a CU's
// few workgroups listed, summed and wrote in turn.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kRun = 8192, kPer = kRun / kSortThreads;  // entries a run, at most a thread
constexpr int kFew = 8;

// four columns of a row, as loaded
template <bool BF16>
struct Four {
  uint32_t w[BF16 ? 2 : 4];
  __device__ __forceinline__ float operator[](int k) const {
    if (!BF16) return __uint_as_float(w[k % (BF16 ? 2 : 4)]);
    return __uint_as_float((k & 1) ? (w[k >> 1] & 0xFFFF0000u) : (w[k >> 1] << 16));
  }
};

template <bool BF16>
__device__ __forceinline__ Four<BF16> load4(const EmbedArgs& p, int64_t t, int64_t col) {
  const int64_t i = t * p.D + col;
  Four<BF16> x;
  if (col + 4 <= p.D) {
    if (BF16) {
      const u32x2_a2 w = *reinterpret_cast<const u32x2_a2*>(static_cast<const uint16_t*>(p.in) + i);
      x.w[0] = w[0];
      x.w[1] = w[1];
    } else {
      const u32x4_a2 w = *reinterpret_cast<const u32x4_a2*>(static_cast<const float*>(p.in) + i);
#pragma unroll
      for (int k = 0; k < (BF16 ? 2 : 4); ++k) x.w[k] = w[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < (BF16 ? 2 : 4); ++k) x.w[k] = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (col + k >= p.D) continue;
      if (BF16)
        x.w[k >> 1] |= (uint32_t) static_cast<const uint16_t*>(p.in)[i + k] << (16 * (k & 1));
      else
        x.w[k % (BF16 ? 2 : 4)] = static_cast<const uint32_t*>(p.in)[i + k];
    }
  }
  return x;
}

__device__ __forceinline__ void store4(const EmbedArgs& p, int64_t row, int64_t col, f32x4_a4 v) {
  float* dst = static_cast<float*>(p.out) + row * p.D + col;
  if (col + 4 <= p.D) {
    *reinterpret_cast<f32x4_a4*>(dst) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + k < p.D) dst[k] = v[k];
  }
}

// the lanes of the wave whose low six bits of `key` are this lane's
__device__ __forceinline__ unsigned long long same_key(uint32_t key) {
  unsigned long long same = ~0ull;
#pragma unroll
  for (int b = 0; b < 6; ++b) {
    const unsigned long long set = __ballot((key >> b) & 1u);
    same &= ((key >> b) & 1u) ? set : ~set;
  }
  return same;
}

// A least-significant-digit radix sort of one run, six bits a pass.  Wave w
// holds the w-th part of the present order, 64 entries at a time: an entry's
// rank among its wave's equal digits is the count before plus the equal lanes
// below.  Tokens outside the table and the entries past T take key V, the
// largest.
__global__ __launch_bounds__(kSortThreads) void k_embed_sort(EmbedArgs p, int bits) {
  __shared__ uint32_t s_key[kRun];
  __shared__ uint16_t s_pos[kRun];
  __shared__ int s_at[kSortWaves][64];  // a wave's entries of each digit, then where they go
  __shared__ uint32_t s_many;           // rows listed
  __shared__ uint16_t s_first[kRun / (kFew + 1)];
  static_assert(kRun / (kFew + 1) <= kSortThreads, "a thread for each listed row");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kRun;
  // a lone run needs no more rounds than its tokens fill; others are merged whole
  const int per = gridDim.x > 1 ? kPer : (int)((p.T + kSortThreads - 1) / kSortThreads);
  const int mine = wave * 64 * per + lane;
  uint32_t key[kPer];
  int pos[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (k >= per) break;
    pos[k] = mine + 64 * k;
    const int64_t t = t0 + pos[k];
    const uint32_t tok = t < p.T ? (uint32_t)p.tok[t] : ~0u;
    key[k] = tok < (uint32_t)p.V ? tok : (uint32_t)p.V;
  }
  if (tid == 0) s_many = 0u;
  if (gridDim.x > 1 && blockIdx.x == 0 && tid == 0) *p.count = 0u;
  for (int shift = 0; shift < bits; shift += 6) {
    s_at[wave][lane] = 0;
    __builtin_amdgcn_wave_barrier();
    int rank[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (k >= per) break;
      const uint32_t d = (key[k] >> shift) & 63u;
      const unsigned long long same = same_key(d);
      const int before = s_at[wave][d];
      __builtin_amdgcn_wave_barrier();
      rank[k] = before + __popcll(same & ((1ull << lane) - 1ull));
      if ((same >> lane) == 1ull) s_at[wave][d] = before + __popcll(same);  // the last of the equal lanes
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    if (wave == 0) {
      int count[kSortWaves], all = 0;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) all += count[w] = s_at[w][lane];
      int sum = all;  // inclusive prefix sum over the digits
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(sum, off);
        if (lane >= off) sum += o;
      }
      int base = sum - all;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        s_at[w][lane] = base;
        base += count[w];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (k >= per) break;
      const int to = s_at[wave][(key[k] >> shift) & 63u] + rank[k];
      s_key[to] = key[k];
      s_pos[to] = (uint16_t)pos[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (k >= per) break;
      key[k] = s_key[mine + 64 * k];
      pos[k] = s_pos[mine + 64 * k];
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (k >= per) break;
    const int at = mine + 64 * k;
    p.sorted[t0 + at] = make_uint2(key[k], (uint32_t)(t0 + pos[k]));
  }
  if (gridDim.x > 1) return;
  // the rows with more than kFew entries (s_key is sorted; padding has key V):
  // where they begin, in any order, then, a thread each, where they end
  const int n = per * kSortThreads;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (k >= per) break;
    const int at = mine + 64 * k;
    const uint32_t row = key[k];
    if (row < p.V && at + kFew < n && s_key[at + kFew] == row && (at == 0 || s_key[at - 1] != row))
      s_first[atomicAdd(&s_many, 1u)] = (uint16_t)at;
  }
  __syncthreads();
  if (tid == 0) *p.count = s_many;
  if (tid >= (int)s_many) return;
  const int first = s_first[tid];
  const uint32_t row = s_key[first];
  int lo = first + kFew + 1, hi = n;
  while (lo < hi) {
    const int m = (lo + hi) / 2;
    if (s_key[m] == row)
      lo = m + 1;
    else
      hi = m;
  }
  p.many[tid] = make_uint2((uint32_t)first, (uint32_t)(lo - first));
}

__global__ __launch_bounds__(kEmbThreads) void k_embed_fill(float* out, int64_t n) {
  const int64_t i = ((int64_t)blockIdx.x * kEmbThreads + threadIdx.x) * 4;
  if (i + 4 <= n) {
    *reinterpret_cast<f32x4_a4*>(out + i) = f32x4_a4{0.f, 0.f, 0.f, 0.f};
  } else {
    for (int64_t e = i; e < n; ++e) out[e] = 0.0f;
  }
}

// Runs of `len` sorted entries of src, merged in pairs into dst: an entry of
// the left run goes past the smaller ones of the right, one of the right run
// past the smaller and equal ones of the left.
__global__ __launch_bounds__(kEmbThreads) void k_embed_merge(const uint2* __restrict__ src, uint2* __restrict__ dst,
                                                             int64_t n, int64_t len) {
  const int64_t i = (int64_t)blockIdx.x * kEmbThreads + threadIdx.x;
  if (i >= n) return;
  const int64_t pair = i / (2 * len) * (2 * len), mid = min(pair + len, n), end = min(pair + 2 * len, n);
  const uint2 e = src[i];
  const bool left = i < mid;
  const int64_t other = left ? mid : pair;
  int64_t lo = other, hi = left ? end : mid;
  while (lo < hi) {
    const int64_t m = (lo + hi) / 2;
    if (src[m].x < e.x || (!left && src[m].x == e.x))
      lo = m + 1;
    else
      hi = m;
  }
  dst[i + (lo - other) - (left ? 0 : mid - pair)] = e;
}

// 2^lpr_log2 lanes an entry, kWide vectors of four columns a lane, two entries
// of the row in flight
constexpr int kWide = 4;
template <bool BF16>
__device__ __forceinline__ void sum_few(const EmbedArgs& p, int lpr_log2, int64_t block, int64_t part, bool list) {
  const int lpr = 1 << lpr_log2, l = threadIdx.x & (lpr - 1);
  const int64_t i = (block * kEmbThreads + threadIdx.x) >> lpr_log2;
  if (i >= p.T) return;
  // entries i - 1 .. i + kFew, all at once
  const uint32_t before = i > 0 ? p.sorted[i - 1].x : ~0u;
  uint2 e[kFew + 1];
#pragma unroll
  for (int k = 0; k <= kFew; ++k) e[k] = i + k < p.T ? p.sorted[i + k] : make_uint2(~0u, 0u);
  const uint32_t row = e[0].x;
  if (row >= p.V || before == row) return;
  if (e[kFew].x == row) {
    if (list && l == 0 && part == 0) {  // the row's end, by bisection
      int64_t lo = i + kFew + 1, hi = p.T;
      while (lo < hi) {
        const int64_t m = (lo + hi) / 2;
        if (p.sorted[m].x == row)
          lo = m + 1;
        else
          hi = m;
      }
      p.many[atomicAdd(p.count, 1u)] = make_uint2((uint32_t)i, (uint32_t)(lo - i));  // (any order will do)
    }
    return;
  }
  const int64_t c0 = part * 4 * kWide * lpr + 4 * l;
  float acc[kWide][4] = {};
#pragma unroll
  for (int q = 0; q < kFew; q += 2) {
    if (e[q].x != row) break;
    const bool two = e[q + 1].x == row;
    Four<BF16> x[kWide], y[kWide];
#pragma unroll
    for (int w = 0; w < kWide; ++w) {
      const int64_t col = c0 + 4 * w * lpr;
      if (col < p.D) x[w] = load4<BF16>(p, e[q].y, col);
      if (col < p.D && two) y[w] = load4<BF16>(p, e[q + 1].y, col);
    }
#pragma unroll
    for (int w = 0; w < kWide; ++w) {
      if (c0 + 4 * w * lpr >= p.D) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[w][j] += x[w][j];
      if (!two) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[w][j] += y[w][j];
    }
  }
#pragma unroll
  for (int w = 0; w < kWide; ++w) {
    const int64_t col = c0 + 4 * w * lpr;
    if (col < p.D)
      store4(p, row, col, f32x4_a4{acc[w][0] * p.scale, acc[w][1] * p.scale, acc[w][2] * p.scale, acc[w][3] * p.scale});
  }
}

// One listed row and 4 * 2^lpr_log2 columns a workgroup at a time: each group
// of lanes sums its part of the row's entries, the first joins the parts.
template <bool BF16>
__device__ __forceinline__ void sum_many(const EmbedArgs& p, int lpr_log2, uint32_t chunks, uint32_t block,
                                         uint32_t blocks, float* s_sum) {
  constexpr int kAhead = 8;  // rows of dout in flight per lane
  const int tid = threadIdx.x, lpr = 1 << lpr_log2;
  const int group = tid >> lpr_log2, groups = kEmbThreads >> lpr_log2;
  const uint64_t tasks = (uint64_t)*p.count * chunks;
  for (uint64_t task = block; task < tasks; task += blocks) {
    const uint2 listed = p.many[task / chunks];
    const int64_t i = listed.x, n = listed.y;
    const int64_t col = ((int64_t)(task % chunks) * lpr + (tid & (lpr - 1))) * 4;
    const bool on = col < p.D;
    const int64_t part = (n + groups - 1) / groups, q0 = i + group * part, q1 = min(q0 + part, i + n);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (on) {
      for (int64_t q = q0; q < q1; q += kAhead) {
        Four<BF16> x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (q + k < q1) x[k] = load4<BF16>(p, p.sorted[q + k].y, col);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (q + k >= q1) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] += x[k][j];
        }
      }
    }
    *reinterpret_cast<f32x4_a4*>(s_sum + 4 * tid) = f32x4_a4{acc[0], acc[1], acc[2], acc[3]};
    __syncthreads();
    if (group == 0 && on) {
      for (int g = 1; g < groups && g * part < n; ++g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += s_sum[4 * ((g << lpr_log2) + tid) + j];
      }
      store4(p, p.sorted[i].x, col, f32x4_a4{acc[0] * p.scale, acc[1] * p.scale, acc[2] * p.scale, acc[3] * p.scale});
    }
    __syncthreads();
  }
}

// How the sums' workgroups are dealt out: `many` of the first row of the grid
// take the listed rows, the others of each row one part of the columns for the
// short rows.
struct SumGrid {
  uint32_t many, chunks;
  int many_log2, few_log2;  // lanes over columns
  bool list;                // the short rows' lanes list the long ones
};

template <bool BF16>
__global__ __launch_bounds__(kEmbThreads) void k_embed_sums(EmbedArgs p, SumGrid g) {
  __shared__ __align__(16) float s_sum[kEmbThreads * 4];
  if (blockIdx.x >= g.many)
    sum_few<BF16>(p, g.few_log2, blockIdx.x - g.many, blockIdx.y, g.list);
  else if (blockIdx.y == 0)
    sum_many<BF16>(p, g.many_log2, g.chunks, blockIdx.x, g.many, s_sum);
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

// Workspace: the sorted entries (twice if runs are merged), the list of rows
// with many entries, its length.
static int64_t sorted_entries(int64_t T) { return (T + kRun - 1) / kRun * kRun; }

int64_t embed_grad_workspace(int64_t T) {
  const int64_t n = sorted_entries(T);
  return T == 0 ? 0 : (n > kRun ? 2 * n : n) * 8 + (T / kFew + 1) * 8 + 8;
}

template <bool BF16>
static void launch_embed_sums(const EmbedArgs& a, bool listed, int cus, hipStream_t st) {
  const int64_t vecs = (a.D + 3) / 4;
  const int lpr = log2_up((vecs + kWide - 1) / kWide, 2, 6);  // lanes that cover a row at once, up to a wave
  const int64_t per = kEmbThreads >> lpr, parts = (vecs + (kWide << lpr) - 1) / (kWide << lpr);
  const int lm = log2_up(vecs, 2, 4);
  const int64_t chunks = (vecs + (1 << lm) - 1) >> lm;
  const uint32_t many = a.T > kFew ? (uint32_t)std::min<int64_t>(a.T / kFew * chunks, 8 * cus) : 0;
  SumGrid g{listed ? many : 0, (uint32_t)chunks, lm, lpr, !listed};
  const dim3 grid((unsigned)(g.many + (a.T + per - 1) / per), (unsigned)parts);
  hipLaunchKernelGGL(k_embed_sums<BF16>, grid, dim3(kEmbThreads), 0, st, a, g);
  if (listed || many == 0) return;
  g.many = many;
  hipLaunchKernelGGL(k_embed_sums<BF16>, dim3(many), dim3(kEmbThreads), 0, st, a, g);
}

void launch_embed_grad(const EmbedArgs& args, void* workspace, int cus, hipStream_t st) {
  EmbedArgs a = args;
  const int64_t n = sorted_entries(a.T), vecs = (a.V * a.D + 3) / 4;
  const int runs = (int)(n / kRun);
  a.sorted = static_cast<uint2*>(workspace);
  uint2* other = a.sorted + n;
  a.many = a.sorted + (n > kRun ? 2 * n : n);
  a.count = reinterpret_cast<uint32_t*>(a.many + a.T / kFew + 1);
  int bits = 1;
  while (a.V >> bits) ++bits;  // keys 0 .. V
  hipLaunchKernelGGL(k_embed_fill, dim3((unsigned)((vecs + kEmbThreads - 1) / kEmbThreads)), dim3(kEmbThreads), 0, st,
                     static_cast<float*>(a.out), a.V * a.D);
  if (a.T == 0) return;
  hipLaunchKernelGGL(k_embed_sort, dim3((unsigned)runs), dim3(kSortThreads), 0, st, a, bits);
  for (int64_t len = kRun; len < n; len *= 2) {
    hipLaunchKernelGGL(k_embed_merge, dim3((unsigned)(n / kEmbThreads)), dim3(kEmbThreads), 0, st, a.sorted, other, n,
                       len);
    std::swap(a.sorted, other);
  }
  if (a.bf16)
    launch_embed_sums<true>(a, runs == 1, cus, st);
  else
    launch_embed_sums<false>(a, runs == 1, cus, st);
}

}  // namespace nvfp4
