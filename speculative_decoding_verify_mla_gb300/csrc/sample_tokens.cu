// sample_tokens.cu - one token per row of logits, drawn under a temperature,
// top-k, top-p and min-p from a given uniform, and the distribution it was
// drawn from.
//
// Definition, for a row x[0..V) with largest logit m (-inf masks a token):
//   w_v = exp((x_v - m) / temperature), tokens with w_v < 2^-40 are left out;
//   top-k keeps x_v >= the k-th largest logit; top-p keeps x_v >= the largest
//   logit s for which the tokens of top-k with x >= s hold at least the share
//   p of top-k's weight; min-p keeps w_v >= min_p.  (Ties at a border are all
//   kept, so each filter is a threshold on the logit.)
//   token = the smallest v with sum_{i<=v, kept} w_i > u * sum_kept w.
//
// Exact sums.  A vocabulary of 1.6e5 tokens of similar weight has steps of
// 6e-6 in its distribution: an error of 1e-7 in a running sum (fp32) would
// change one draw in thirty, and the result would depend on the order of
// summation.  So a weight is a fixed-point integer (relative error below
// 2^-30; the unit is as small as lets V of them stay below 2^63) and all sums
// are 64-bit integers: they are associative, and the token is a function of
// the inputs alone.  The weight is
// 2^t with t = x * log2(e)/temperature carried as an unevaluated fp32 pair,
// split as t = k/256 + g with integer k; 2^(k/256) comes from a table of 256
// integers and 2^g - 1, |g| <= 1/512, from three Taylor terms (the table
// method of Tang 1989).
//
// One thread-block cluster per row; each CTA keeps its slice of the row in
// shared memory, so the logits cross HBM once whatever the filters need.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "sv_cluster.cuh"
#include "sv_ptx.cuh"

namespace sv {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterMax = 8;
constexpr int kSupportBits = 40;     // weights below 2^-40 of the largest are left out
constexpr int kMaxVocab = 1 << 22;   // leaves a weight 41 bits
constexpr float kCoarseMax = 8192.f;  // |x| log2(e)/temperature up to which the row needs no shift

// round(2^31 2^(j/256)), j = 0..255, by the exponential series.
struct Exp2Table {
  uint32_t v[256];
  constexpr Exp2Table() : v() {
    for (int j = 0; j < 256; ++j) {
      const double y = j * 0.693147180559945309417232121458 / 256.0;
      double term = 1.0, sum = 1.0;
      for (int i = 1; i < 24; ++i) {
        term *= y / i;
        sum += term;
      }
      v[j] = (uint32_t)(sum * 2147483648.0 + 0.5);
    }
  }
};
__device__ constexpr Exp2Table kExp2{};

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {  // exact: the values are bf16
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

struct SampleArgs {
  const void* logits;
  const float *uniforms, *temperature, *top_p, *min_p;  // per-row arrays, or NULL for the *_all value
  const int32_t* top_k;
  float temperature_all, top_p_all, min_p_all;
  int top_k_all;
  long long row_stride;
  int V, slice;  // slice: logits per CTA, a multiple of 8
  int down;      // the largest weight is mant << 31 >> down (mant < 2^32): V of them stay below 2^63
  int32_t* tokens;
  float* probs;
  int32_t* status;
};

struct Shared {
  uint32_t table[256];
  u64 slot[2][kClusterMax];
  u64 warp_sum[kWarps];
  u64 block;
  int token;
};

// The weight function of a row, 2^((x - base) c).
struct RowWeight {
  float base, ch, cl;  // c = ch + cl
  int top;             // exponent of the largest weight, + down
};
struct Weight {
  uint32_t mant;  // [2^31, 2^32)
  int shift;      // the weight is (mant << 31) >> shift
};
__device__ __forceinline__ int grid256(float p, float* grid) {
  // p rounded to a multiple of 1/256: adding 1.5 * 2^15 leaves 8 fraction bits
  const float k = p + 49152.f;
  *grid = k - 49152.f;
  return (int)(__float_as_uint(k) - __float_as_uint(49152.f));
}
__device__ __forceinline__ Weight weight_of(const RowWeight& rw, const uint32_t* table, float x) {
  const float d = x - rw.base;
  const float p = d * rw.ch;
  const float e = fmaf(d, rw.cl, fmaf(d, rw.ch, -p));
  const float pc = fmaxf(p, -12000.f);  // far below every weight that counts; also -inf and NaN
  float grid;
  const int k = grid256(pc, &grid);
  const float g = (pc - grid) + e;
  // 2^g - 1
  const float r = g * fmaf(g, fmaf(g, 0.0555041087f, 0.2402265070f), 0.6931471806f);
  Weight w;
  const uint32_t t = table[k & 255];
  w.mant = t + (uint32_t)__float2int_rn((float)t * r);
  w.shift = min(rw.top - (k >> 8), 63);
  return w;
}
// The lowest bit is always set: like a rounding, unlike the cut alone, that
// is right on average, so the sum of many small weights does not drift.
__device__ __forceinline__ u64 fixed(const Weight& w) { return (((u64)w.mant << 31) >> w.shift) | 1; }

// Order-preserving integer of a float, and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// floor(f 2^64) of f in [0, 1]; 1 and above give 2^64 - 1, NaN and below 0 give 0.
__device__ __forceinline__ u64 fraction64(float f) {
  if (!(f > 0.f)) return 0;
  if (f >= 1.f) return ~0ull;
  return (u64)((double)f * 18446744073709551616.0);
}

// Sums and maxima over the cluster; every thread gets the result.
struct Cluster {
  Shared* s;
  uint32_t rank, size;
  int parity;

  __device__ __forceinline__ u64 block_sum(u64 v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) s->warp_sum[warp] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s->warp_sum[w];
    __syncthreads();
    return v;
  }
  // mine: the CTA's number, the same in every thread
  __device__ __forceinline__ void exchange(u64 mine) {
    if (threadIdx.x < size) cluster_st64(cluster_map(&s->slot[parity][rank], threadIdx.x), mine);
    cluster_sync();
  }
  __device__ __forceinline__ u64 sum(u64 v, u64* before = nullptr) {
    exchange(block_sum(v));
    u64 a = 0, b = 0;
    for (uint32_t r = 0; r < size; ++r) {
      if (r < rank) b += s->slot[parity][r];
      a += s->slot[parity][r];
    }
    if (before) *before = b;
    parity ^= 1;
    return a;
  }
  __device__ __forceinline__ float max(float v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (lane == 0) s->warp_sum[warp] = __float_as_uint(v);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v = fmaxf(v, __uint_as_float((uint32_t)s->warp_sum[w]));
    __syncthreads();
    exchange(__float_as_uint(v));
    for (uint32_t r = 0; r < size; ++r) v = fmaxf(v, __uint_as_float((uint32_t)s->slot[parity][r]));
    parity ^= 1;
    return v;
  }
};

// The CTA's slice of the row as groups of 16 aligned bytes; element i of group
// g is logit g * kN - head + i of the slice, -inf where that is outside it.
template <typename T>
struct Slice {
  static constexpr int kN = Vec<T>::kN;
  const T* src;   // the slice's first logit in global memory
  uint4* stage;   // its groups in shared memory (resident rows)
  int n, head, groups;

  __device__ __forceinline__ uint4 fetch(int g) const {
    const int e0 = g * kN - head;
    if (e0 >= 0 && e0 + kN <= n) {
      uint4 v;
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "l"(src + e0));
      return v;
    }
    float x[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = e0 + i >= 0 && e0 + i < n ? Vec<T>::one(src + e0 + i) : -INFINITY;
    return Vec<T>::pack(x);
  }
  template <bool kResident>
  __device__ __forceinline__ void load(int g, float (&x)[kN]) const {
    Vec<T>::unpack(kResident ? stage[g] : fetch(g), x);
  }
  // f(x, logit of the slice) over this thread's groups: a warp owns a run of
  // consecutive groups, its lanes neighbouring ones
  __device__ __forceinline__ int warp_groups() const { return (groups + kWarps - 1) / kWarps; }
  template <bool kResident, class F>
  __device__ __forceinline__ void each(F f) const {
    const int per = warp_groups(), warp = threadIdx.x >> 5;
    const int end = min(groups, (warp + 1) * per);
#pragma unroll 2
    for (int g = warp * per + (threadIdx.x & 31); g < end; g += 32) {
      float x[kN];
      load<kResident>(g, x);
#pragma unroll
      for (int i = 0; i < kN; ++i) f(x[i], g * kN - head + i);
    }
  }
};

template <typename T, bool kResident>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint4 s_stage[];
  __shared__ Shared s;
  constexpr int kN = Vec<T>::kN;
  Cluster cl{&s, cluster_rank(), cluster_size(), 0};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = (int)(blockIdx.x / cl.size);
  const long long lo = (long long)cl.rank * a.slice;
  Slice<T> sl;
  sl.src = static_cast<const T*>(a.logits) + t * a.row_stride + lo;
  sl.stage = s_stage;
  sl.n = (int)max(0ll, min((long long)a.slice, a.V - lo));
  sl.head = (int)((reinterpret_cast<uintptr_t>(sl.src) & 15u) / sizeof(T));
  sl.groups = sl.n > 0 ? (sl.head + sl.n + kN - 1) / kN : 0;
  if (threadIdx.x < 256) s.table[threadIdx.x] = kExp2.v[threadIdx.x];

  // the row's settings
  const float u = __ldg(a.uniforms + t);
  float tau = a.temperature ? __ldg(a.temperature + t) : a.temperature_all;
  float top_p = a.top_p ? __ldg(a.top_p + t) : a.top_p_all;
  float min_p = a.min_p ? __ldg(a.min_p + t) : a.min_p_all;
  int top_k = a.top_k ? __ldg(a.top_k + t) : a.top_k_all;

  // largest logit (fmaxf passes over NaN)
  float m = -INFINITY;
  {
    const int per = sl.warp_groups(), end = min(sl.groups, (warp + 1) * per);
#pragma unroll 4
    for (int g = warp * per + lane; g < end; g += 32) {
      const uint4 v = sl.fetch(g);
      if (kResident) s_stage[g] = v;
      float x[kN];
      Vec<T>::unpack(v, x);
#pragma unroll
      for (int i = 0; i < kN; ++i) m = fmaxf(m, x[i]);
    }
  }
  cluster_sync();  // every CTA of the cluster runs
  m = cl.max(m);
  float* const probs = a.probs ? a.probs + (long long)t * a.V + lo : nullptr;
  if (!(fabsf(m) < INFINITY) || !(tau < INFINITY)) {
    // nothing to draw from: no finite largest logit, or no temperature
    if (probs)
      for (int i = threadIdx.x; i < sl.n; i += kThreads) probs[i] = 0.f;
    if (cl.rank == 0 && threadIdx.x == 0) {
      a.tokens[t] = -1;
      if (a.status) atomicOr(a.status, SV_DEV_BAD_LOGITS);
    }
    return;
  }

  const bool greedy = tau < 5.4210109e-20f;  // 2^-64
  if (greedy) {
    tau = 1.f;
    top_k = 0;
    top_p = 1.f;
    min_p = 1.f;
  }
  // t = x log2(e)/temperature as a pair; rows with large |t| are shifted by
  // their largest logit (there x - m is exact wherever the weight counts:
  // |x - m| is then below a hundredth of |m|)
  RowWeight rw;
  {
    const double c = 1.4426950408889634074 / (double)tau;
    rw.ch = (float)c;
    rw.cl = (float)(c - (double)rw.ch);
    rw.base = fabsf(m * rw.ch) < kCoarseMax ? 0.f : m;
    float grid;
    rw.top = (grid256((m - rw.base) * rw.ch, &grid) >> 8) + a.down;
  }
  // the threshold so far: the support, and min-p
  float theta;
  {
    const double ln_floor = min_p >= 1.f ? 0.0 : (min_p > 0.f ? log((double)min_p) : -1e300);
    const double support = -kSupportBits * 0.69314718055994530942;
    theta = __double2float_ru((double)m + (double)tau * fmax(ln_floor, support));
    theta = fminf(theta, m);
  }

  // top-k: the largest key that at least k logits reach
  float theta_k = __double2float_ru((double)m - (double)tau * (kSupportBits * 0.69314718055994530942));
  if (top_k > 0 && top_k < a.V) {
    uint32_t lo_k = key_of(-INFINITY), hi_k = key_of(m);
    while (lo_k < hi_k) {
      const uint32_t mid = lo_k + (hi_k - lo_k) / 2 + 1;
      const float v = key_float(mid);
      unsigned cnt = 0;
      sl.template each<kResident>([&](float x, int) { cnt += x >= v; });
      if (cl.sum(cnt) >= (u64)top_k)
        lo_k = mid;
      else
        hi_k = mid - 1;
    }
    theta_k = fmaxf(theta_k, key_float(lo_k));
    theta = fmaxf(theta, theta_k);
  }
  // top-p: the largest key whose logits hold the share p of top-k's weight
  if (top_p < 1.f) {
    auto mass_from = [&](float v) {
      u64 w = 0;
      sl.template each<kResident>([&](float x, int) {
        if (x >= v) w += fixed(weight_of(rw, s.table, x));
      });
      return cl.sum(w);
    };
    const u64 all = mass_from(theta_k), f = fraction64(top_p);
    const u64 need = __umul64hi(f, all) + (f * all != 0 ? 1 : 0);  // the least integer that is p of all, or more
    uint32_t lo_k = key_of(theta_k), hi_k = key_of(m);
    while (lo_k < hi_k) {
      const uint32_t mid = lo_k + (hi_k - lo_k) / 2 + 1;
      if (mass_from(fmaxf(theta_k, key_float(mid))) >= need)
        lo_k = mid;
      else
        hi_k = mid - 1;
    }
    theta = fmaxf(theta, key_float(lo_k));
  }

  // the draw, in the order of the vocabulary
  u64 mine = 0;
  sl.template each<kResident>([&](float x, int) {
    if (x >= theta) mine += fixed(weight_of(rw, s.table, x));
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
  u64 before, total;
  total = cl.sum(lane == 0 ? mine : 0, &before);
  // block_sum left every warp's sum in warp_sum
  const u64 target = greedy ? 0 : min(__umul64hi(fraction64(u), total), total - 1);
  for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
  if (target >= before && target - before < mine) {
    // this warp holds the token
    const int per = sl.warp_groups(), end = min(sl.groups, (warp + 1) * per);
    u64 run = before;
    for (int g0 = warp * per; g0 < end; g0 += 32) {
      const int g = g0 + lane;
      float x[kN];
      u64 w[kN], sum = 0;
      if (g < end) {
        sl.template load<kResident>(g, x);
      } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        w[i] = x[i] >= theta ? fixed(weight_of(rw, s.table, x[i])) : 0;
        sum += w[i];
      }
      u64 incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
      }
      const u64 upto = run + incl - sum;
      if (target >= upto && target < upto + sum) {
        u64 c = upto;
        int hit = -1;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          c += w[i];
          if (hit < 0 && c > target) hit = i;
        }
        const int token = (int)(lo + g * kN - sl.head + hit);
        a.tokens[t] = token;
        for (uint32_t r = 0; r < cl.size; ++r) cluster_st(cluster_map(&s.token, r), (uint32_t)token);
      }
      run += __shfl_sync(0xFFFFFFFFu, incl, 31);
      if (run > target) break;
    }
  }
  cluster_sync();
  if (!probs) return;
  const float inv = (float)(1.0 / (double)total);
  if (greedy) {
    for (int i = threadIdx.x; i < sl.n; i += kThreads) probs[i] = lo + i == s.token ? 1.f : 0.f;
    return;
  }
  sl.template each<kResident>([&](float x, int i) {
    if (i < 0 || i >= sl.n) return;
    float p = 0.f;
    if (x >= theta) {
      const Weight w = weight_of(rw, s.table, x);
      p = (float)w.mant * __uint_as_float((uint32_t)(127 + 31 - w.shift) << 23) * inv;
    }
    probs[i] = p;
  });
}

// ------------------------------------------------------------------ host side
constexpr size_t kStageTwo = 96 * 1024;   // two CTAs of an SM keep their slices
constexpr size_t kStageOne = 208 * 1024;  // one CTA does

struct Shape {
  int ctas, slice;
  size_t stage;  // bytes of a resident slice, 0: rows are read again for every pass
};
// The fewest CTAs a row whose slices fit two to an SM; more where few rows
// would leave SMs idle (a row's passes get shorter, down to 4096 logits a CTA).
Shape row_shape(int T, int V, int elem) {
  Shape sh;
  auto slice_of = [&](int c) { return (int)((((long long)V + c - 1) / c + 7) / 8 * 8); };
  auto stage_of = [&](int c) { return ((size_t)slice_of(c) * elem + 16 + 15) / 16 * 16; };
  int c = 1;
  while (c < kClusterMax && stage_of(c) > kStageTwo) c *= 2;
  while (c < kClusterMax && (long long)T * c < 304 && slice_of(2 * c) >= 4096) c *= 2;
  sh.ctas = c;
  sh.slice = slice_of(c);
  sh.stage = stage_of(c) <= kStageOne ? stage_of(c) : 0;
  return sh;
}

template <typename T, bool kResident>
cudaError_t launch_sample(const SampleArgs& a, int rows, const Shape& sh, cudaStream_t st) {
  auto kernel = sample_kernel<T, kResident>;
  if (kResident) {
    static std::atomic<bool> done[64];  // per instance and device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kStageOne);
      if (e != cudaSuccess) return e;
      if (dev < 64) done[dev].store(true, std::memory_order_release);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * sh.ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kResident ? sh.stage : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)sh.ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

inline bool off_by(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace
}  // namespace sv

extern "C" sv_status sample_tokens(const void* logits, int logits_type, int T, int V, long long row_stride,
                                   const float* uniforms, const float* temperature, float temperature_all,
                                   const int32_t* top_k, int top_k_all, const float* top_p, float top_p_all,
                                   const float* min_p, float min_p_all, int32_t* tokens, float* probs,
                                   int32_t* status, sv_stream_t stream) {
  using namespace sv;
  if (T < 0) return SV_ERR_SHAPE;
  if (logits_type != SV_LOGITS_F32 && logits_type != SV_LOGITS_BF16) return SV_ERR_UNSUPPORTED;
  if (T == 0) return SV_OK;
  if (V < 1 || row_stride < V || T > 0x7FFFFFFF / kClusterMax) return SV_ERR_SHAPE;
  if (V > kMaxVocab) return SV_ERR_UNSUPPORTED;
  if (!temperature && !(temperature_all < INFINITY)) return SV_ERR_SHAPE;
  if ((!top_p && top_p_all != top_p_all) || (!min_p && min_p_all != min_p_all)) return SV_ERR_SHAPE;
  if (!logits || !uniforms || !tokens) return SV_ERR_NULL;
  const int elem = logits_type == SV_LOGITS_F32 ? 4 : 2;
  if (off_by(logits, elem) || off_by(uniforms, 4) || off_by(tokens, 4) || off_by(probs, 4) || off_by(temperature, 4) ||
      off_by(top_k, 4) || off_by(top_p, 4) || off_by(min_p, 4))
    return SV_ERR_ALIGN;
  SampleArgs a;
  a.logits = logits;
  a.uniforms = uniforms;
  a.temperature = temperature;
  a.top_p = top_p;
  a.min_p = min_p;
  a.top_k = top_k;
  a.temperature_all = temperature_all;
  a.top_p_all = top_p_all;
  a.min_p_all = min_p_all;
  a.top_k_all = top_k_all;
  a.row_stride = row_stride;
  a.V = V;
  a.tokens = tokens;
  a.probs = probs;
  a.status = status;
  const Shape sh = row_shape(T, V, elem);
  a.slice = sh.slice;
  a.down = 0;
  while ((1 << a.down) < V) ++a.down;  // V <= 2^down: V (2^63 >> down) <= 2^63
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (elem == 4)
    e = sh.stage ? launch_sample<float, true>(a, T, sh, st) : launch_sample<float, false>(a, T, sh, st);
  else
    e = sh.stage ? launch_sample<__nv_bfloat16, true>(a, T, sh, st) : launch_sample<__nv_bfloat16, false>(a, T, sh, st);
  if (e == cudaSuccess) return SV_OK;
  cudaGetLastError();
  return SV_ERR_LAUNCH;
}
