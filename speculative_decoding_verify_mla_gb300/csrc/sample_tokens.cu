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
// shared memory, so the logits cross HBM once whatever the filters need, and
// the CTAs meet in distributed shared memory.  How the thresholds are found:
//  * A small top-k (the usual one): every warp publishes its largest logits;
//    the k-th largest of those bounds the k-th largest of the row from below
//    and leaves about 1.4 k candidates, which one CTA ranks; top-p, min-p and
//    the draw then look at the candidates alone.
//  * A large top-k, or top-p over the whole vocabulary: a histogram of counts
//    over 1/64 octaves of weight.  Counts place the k-th logit exactly; for
//    top-p they place the border to within a few bins, then one pass sums the
//    weight above those bins and the whole weight exactly and collects what is
//    inside, which one CTA ranks.
//  * Where a bin holds too many (ties): bisection over the logits' bits.
#include <atomic>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

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
constexpr float kHottest = 1.2676506e30f;  // 2^100: beyond, 1/temperature loses bits
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
  double ln_min_p_all;  // ln(min_p_all), 0 above 1
  long long row_stride;
  int V, slice;  // slice: logits per CTA, a multiple of 8
  int down;      // the largest weight is mant << 31 >> down (mant < 2^32): V of them stay below 2^63
  int32_t* tokens;
  float* probs;
  int32_t* status;
};

constexpr int kBins = 2592;       // bins of 1/64 octave of weight: 40.5 octaves, a multiple of 8 shares
constexpr int kList = 512;        // candidates that one CTA ranks, one per thread
constexpr int kPublished = 512;
constexpr int kTries = 2;         // guesses of the top-p border before the bisection

struct Shared {
  uint32_t table[256];
  u64 slot[2][3][kClusterMax];     // exchange: parity, value, rank
  u64 warp_sum[3][kWarps];
  __align__(16) uint32_t pub[kPublished];  // largest keys of every warp of the cluster
  __align__(16) u64 cand[kList];   // key << 32 | index
  int count;                       // candidates found here
  int token;
  uint32_t found;                  // a key, or a bin
  int bins[2];
  u64 before[3];                   // of the bin found: logits before and in it; at the window's start: weight
  float delta[2];
  __align__(16) u64 list[kList], sorted[kList];
  uint32_t hist[kBins];            // see bin_estimate
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
  const uint32_t b = __float_as_uint(f);
  const int e = (int)(b >> 23) - 86;  // mantissa * 2^(exponent - 150 + 64)
  const u64 mant = (b & 0x7FFFFFu) | 0x800000u;
  return e >= 0 ? mant << e : (e > -24 ? mant >> -e : 0);
}
// The least integer that is the fraction f / 2^64 of v, or more.
__device__ __forceinline__ u64 share_of(u64 f, u64 v) { return __umul64hi(f, v) + (f * v != 0 ? 1 : 0); }

// Sums and maxima over the CTA and the cluster; every thread gets the result.
struct Cluster {
  Shared* s;
  uint32_t rank, size;
  int parity;

  __device__ __forceinline__ void sync() const {
    if (size == 1)
      __syncthreads();
    else
      cluster_sync();
  }
  template <int kValues>
  __device__ __forceinline__ void block_sum(u64 (&v)[kValues]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
      if (lane == 0) s->warp_sum[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      v[i] = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v[i] += s->warp_sum[i][w];
    }
  }
  // Every CTA's values to every CTA; returns this exchange's slots
  // [value][rank].  v: the same in every thread.  Slots alternate: a CTA can
  // be one exchange ahead of a reader, not two.
  template <int kValues>
  __device__ __forceinline__ const u64 (*exchange(const u64 (&v)[kValues]))[kClusterMax] {
    u64(*const to)[kClusterMax] = s->slot[parity];
    parity ^= 1;
    if (threadIdx.x < size) {
#pragma unroll
      for (int i = 0; i < kValues; ++i) cluster_st64(cluster_map(&to[i][rank], threadIdx.x), v[i]);
    }
    sync();
    return to;
  }
  template <int kValues>
  __device__ __forceinline__ const u64 (*sum(u64 (&v)[kValues]))[kClusterMax] {
    block_sum(v);
    const u64(*const all)[kClusterMax] = exchange(v);
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      v[i] = 0;
      for (uint32_t r = 0; r < size; ++r) v[i] += all[i][r];
    }
    return all;
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if ((threadIdx.x & 31) == 0) s->warp_sum[0][threadIdx.x >> 5] = v;
    __syncthreads();
    u64 m[1] = {0};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m[0] = s->warp_sum[0][w] > m[0] ? s->warp_sum[0][w] : m[0];
    const u64(*const all)[kClusterMax] = exchange(m);
    for (uint32_t r = 0; r < size; ++r) m[0] = all[0][r] > m[0] ? all[0][r] : m[0];
    return (uint32_t)m[0];
  }
  // inclusive prefix sum over the CTA in thread order
  __device__ __forceinline__ u64 scan(u64 v, u64* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) s->warp_sum[0][warp] = v;
    __syncthreads();
    u64 all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) v += s->warp_sum[0][w];
      all += s->warp_sum[0][w];
    }
    *total = all;
    return v;
  }
};

__device__ __forceinline__ u64 cluster_ld64(const void* p, uint32_t r) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_map(p, r)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_ld(const void* p, uint32_t r) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_map(p, r)) : "memory");
  return v;
}

// list[0..n) (distinct, padded with zeros to kList) in descending order into
// out[0..n): every entry's rank is counted by a group of threads.
__device__ __forceinline__ void sort_list(const u64* list, u64* out, int n) {
  int per = 1;
  while (per < 32 && 2 * per * n <= kThreads) per *= 2;
  const int i = (int)threadIdx.x / per, part = (int)threadIdx.x & (per - 1);
  const u64 mine = list[i];
  int above = 0;
  for (int j = 2 * part; j < n; j += 2 * per) {
    const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(list + j);
    above += (o.x > mine) + (o.y > mine);
  }
  for (int o = per >> 1; o > 0; o >>= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
  if (i < n && part == 0) out[above] = mine;
  __syncthreads();
}

// The k-th largest of keys[0..n) (n a multiple of 16, k <= n) into *out.
__device__ __forceinline__ void kth_key(const uint32_t* keys, int n, int k, uint32_t* out) {
  int per = 1;
  while (per < 32 && 2 * per * n <= kThreads) per *= 2;
  const int i = (int)threadIdx.x / per, part = (int)threadIdx.x & (per - 1);
  const uint32_t mine = i < n ? keys[i] : 0;
  int above = 0, equal = 0;
  for (int j = 4 * part; j < n; j += 4 * per) {
    const uint4 o = *reinterpret_cast<const uint4*>(keys + j);
    above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
    equal += (o.x == mine) + (o.y == mine) + (o.z == mine) + (o.w == mine);
  }
  for (int o = per >> 1; o > 0; o >>= 1) {
    above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
    equal += __shfl_xor_sync(0xFFFFFFFFu, equal, o);
  }
  if (i < n && above < k && k <= above + equal) *out = mine;  // equal keys write the same
  __syncthreads();
}

// A bin's word: the logits in it (up to 2^22) and, in the upper 9 bits, the sum
// of their places 0..15 in the bin, which is right for up to 32 of them.
constexpr int kCountBits = 23;
constexpr uint32_t kCountMask = (1u << kCountBits) - 1;
// (2 places + 1) / 32 of a bin below its edge: a share of 2^(1/64) - 1 of 88/2^13 per bin
__device__ __forceinline__ u64 bin_estimate(uint32_t word, u64 edge) {
  const u64 c = word & kCountMask;
  const u64 places = c <= 32 ? word >> kCountBits : (15 * c) / 2;
  return c * edge - (edge >> 18) * (2 * places + c) * 88;
}

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

// m + (hi + lo) rounded up to fp32 (the sum's error by Knuth's two-sum), at
// most m and never -inf.
__device__ __forceinline__ float add_up(float m, float hi, float lo) {
  const float s = m + hi;
  const float v = s - m;
  const float t = ((m - (s - v)) + (hi - v)) + lo;
  float r = s + t;
  if (t - (r - s) > 0.f) r = nextafterf(r, INFINITY);
  return fminf(fmaxf(r, -3.402823466e38f), m);
}

template <typename T, bool kResident>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint4 s_stage[];
  __shared__ Shared s;
  constexpr int kN = Vec<T>::kN;
  Cluster cl{&s, cluster_rank(), cluster_size(), 0};
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // waited for before the first exchange
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = (int)(blockIdx.x / cl.size);
  const long long lo = (long long)cl.rank * a.slice;
  Slice<T> sl;
  sl.src = static_cast<const T*>(a.logits) + t * a.row_stride + lo;
  sl.stage = s_stage;
  sl.n = (int)max(0ll, min((long long)a.slice, a.V - lo));
  sl.head = (int)((reinterpret_cast<uintptr_t>(sl.src) & 15u) / sizeof(T));
  sl.groups = sl.n > 0 ? (sl.head + sl.n + kN - 1) / kN : 0;

  // the row's settings
  const float u = __ldg(a.uniforms + t);
  float tau = a.temperature ? __ldg(a.temperature + t) : a.temperature_all;
  float top_p = a.top_p ? __ldg(a.top_p + t) : a.top_p_all;
  float min_p = a.min_p ? __ldg(a.min_p + t) : a.min_p_all;
  int top_k = a.top_k ? __ldg(a.top_k + t) : a.top_k_all;

  // largest logit of the thread (fmaxf passes over NaN)
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
  if (threadIdx.x < 256) s.table[threadIdx.x] = kExp2.v[threadIdx.x];
  const bool greedy = tau < 5.4210109e-20f;  // 2^-64
  if (greedy) {
    tau = 1.f;
    top_k = 0;
    top_p = 1.f;
    min_p = 1.f;
  }
  if (top_k >= a.V) top_k = 0;
  if (min_p > 0.f && threadIdx.x == 0) {
    // the distance from m at which min-p cuts, as a pair
    const double ln = min_p >= 1.f ? 0.0 : (a.min_p ? log((double)min_p) : a.ln_min_p_all);
    const double d = (double)tau * fmax(ln, -kSupportBits * 0.69314718055994530942);
    s.delta[0] = (float)d;
    s.delta[1] = (float)(d - (double)(float)d);
  }
  if (threadIdx.x == 0) s.count = 0;

  // A small top-k looks at the largest logits of every warp, at least twice as
  // many as it asks for (measured: with fewer the candidates behind the bound
  // grow faster than the ranking shrinks).
  int rounds = 0;
  if (top_k > 0) {
    rounds = 1;
    while (rounds < 8 && kWarps * (int)cl.size * rounds < 2 * top_k) rounds *= 2;
    if (kWarps * (int)cl.size * rounds < 2 * top_k || kWarps * (int)cl.size * rounds > kPublished) rounds = 0;
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA of the cluster runs
  float bound = -INFINITY;  // at least top_k logits reach it
  if (rounds > 0) {
    uint32_t key = key_of(m);
    const int mine = ((int)cl.rank * kWarps + warp) * rounds;
    for (int i = 0; i < rounds; ++i) {
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, key);
      if (lane < (int)cl.size) cluster_st(cluster_map(&s.pub[mine + i], lane), top);
      const unsigned who = __ballot_sync(0xFFFFFFFFu, key == top);
      if (lane == __ffs(who) - 1) key = 0;
    }
    cl.sync();
    const int n = kWarps * (int)cl.size * rounds;
    uint32_t top = 0;
    for (int i = lane; i < n; i += 32) top = max(top, s.pub[i]);
    m = key_float(__reduce_max_sync(0xFFFFFFFFu, top));
    kth_key(s.pub, n, top_k, &s.found);
    bound = key_float(s.found);
  } else {
    m = key_float(cl.max(key_of(m)));
  }
  float* const probs = a.probs ? a.probs + (long long)t * a.V + lo : nullptr;
  if (!(fabsf(m) < INFINITY) || !(tau <= kHottest)) {
    // nothing to draw from: no finite largest logit, or no temperature
    if (probs)
      for (int i = threadIdx.x; i < sl.n; i += kThreads) probs[i] = 0.f;
    if (cl.rank == 0 && threadIdx.x == 0) {
      a.tokens[t] = -1;
      if (a.status) atomicOr(a.status, SV_DEV_BAD_LOGITS);
    }
    return;
  }

  // t = x log2(e)/temperature as a pair; rows with large |t| are shifted by
  // their largest logit (there x - m is exact wherever the weight counts:
  // |x - m| is then below a hundredth of |m|)
  RowWeight rw;
  int top_grid;
  {
    // log2(e) = 1.44269502 + 1.92596299e-8
    rw.ch = __fdiv_rn(1.44269502f, tau);
    rw.cl = (fmaf(-rw.ch, tau, 1.44269502f) + 1.92596299e-8f) / tau;
    rw.base = fabsf(m * rw.ch) < kCoarseMax ? 0.f : m;
    float grid;
    top_grid = grid256((m - rw.base) * rw.ch, &grid);
    rw.top = (top_grid >> 8) + a.down;
  }
  // the support ends 40 ln 2 temperatures below m
  float base, theta;
  {
    constexpr double kWidth = kSupportBits * 0.69314718055994530942;
    constexpr float kHi = (float)kWidth, kLo = (float)(kWidth - (double)kHi);
    const float hi = tau * kHi;
    base = add_up(m, -hi, -(fmaf(tau, kHi, -hi) + tau * kLo));
    theta = min_p > 0.f ? fmaxf(base, add_up(m, s.delta[0], s.delta[1])) : base;
  }
  auto weight = [&](float x) { return fixed(weight_of(rw, s.table, x)); };
  auto grid_of = [&](float x, float* off) {
    const float p = fmaxf((x - rw.base) * rw.ch, -12000.f);
    float grid;
    const int k = grid256(p, &grid);
    *off = p - grid;
    return top_grid - k;
  };
  auto collect = [&](float x, int i) {
    const int at = atomicAdd(&s.count, 1);
    if (at < kList) s.cand[at] = ((u64)key_of(x) << 32) | (uint32_t)(lo + i);
  };
  // the cluster's candidates, n <= kList of them, into s.list
  auto bring = [&](const u64* counts, int n) {
    u64 v = 0;
    if ((int)threadIdx.x < n) {
      int at = (int)threadIdx.x;
      uint32_t r = 0;
      while (at >= (int)counts[r]) at -= (int)counts[r++];
      v = cluster_ld64(&s.cand[at], r);
    }
    s.list[threadIdx.x] = v;
    __syncthreads();
  };
  const u64 share = fraction64(top_p), chance = greedy ? 0 : fraction64(u);
  u64 total = 0;

  bool done = false;
  if (bound > -INFINITY) {
    // ---- small top-k: the candidates decide
    sl.template each<kResident>([&](float x, int i) {
      if (x >= bound) collect(x, i);
    });
    __syncthreads();
    u64 mine[1] = {(u64)s.count};
    const u64(*const counts)[kClusterMax] = cl.exchange(mine);
    int n = 0;
    for (uint32_t r = 0; r < cl.size; ++r) n += (int)counts[0][r];
    done = n <= kList;
    if (done && (probs || cl.rank == 0)) {
      bring(counts[0], n);
      sort_list(s.list, s.sorted, n);
      const u64 c = (int)threadIdx.x < n ? s.sorted[threadIdx.x] : 0;
      const float x = c ? key_float((uint32_t)(c >> 32)) : -INFINITY;
      const float x_k = key_float((uint32_t)(s.sorted[top_k - 1] >> 32));
      theta = fmaxf(theta, x_k);
      const u64 w = x >= fmaxf(base, x_k) ? weight(x) : 0;
      if (top_p < 1.f) {
        u64 all;
        const u64 upto = cl.scan(w, &all);
        const u64 need = max(share_of(share, all), 1ull);
        if (upto >= need && upto - w < need) s.found = (uint32_t)(c >> 32);
        __syncthreads();
        theta = fmaxf(theta, key_float(s.found));
      }
      // the kept ones, the first `kept` of the list, in the order of the vocabulary
      const bool keep = x >= theta;
      const int kept = __syncthreads_count(keep);
      u64* const weights = reinterpret_cast<u64*>(s.hist);
      weights[threadIdx.x] = w;
      s.list[threadIdx.x] = keep ? ((u64)(0x7FFFFFFFu - (uint32_t)c) << 32) | threadIdx.x : 0;
      __syncthreads();
      sort_list(s.list, s.sorted, kept);
      const u64 o = (int)threadIdx.x < kept ? s.sorted[threadIdx.x] : 0;
      const u64 w_o = (int)threadIdx.x < kept ? weights[(uint32_t)o] : 0;
      const u64 upto = cl.scan(w_o, &total);
      const u64 target = min(__umul64hi(chance, total), total - 1);
      if (cl.rank == 0 && upto > target && upto - w_o <= target) a.tokens[t] = (int)(0x7FFFFFFFu - (uint32_t)(o >> 32));
    }
  }
  if (!done) {
    // ---- thresholds over the whole row: top-k, then top-p of what it leaves
    for (int kind = 0; kind < 2; ++kind) {
      const bool by_weight = kind == 1;
      if (by_weight ? !(top_p < 1.f) : top_k <= 0) continue;
      __syncthreads();
      for (int b = threadIdx.x; b < kBins; b += kThreads) s.hist[b] = 0;
      __syncthreads();
      sl.template each<kResident>([&](float x, int) {
        if (x >= base) {
          float off;
          const int d = grid_of(x, &off);
          const int place = ((d & 3) << 2) + min((int)(2.f - off * 1024.f), 3);
          atomicAdd(s.hist + (d >> 2), 1u + ((uint32_t)place << kCountBits));
        }
      });
      cl.sync();
      // CTA r adds up share r of the bins (from the largest weights down) and
      // leaves the sums in its own histogram, where no other CTA reads in this phase
      const int own = kBins / (int)cl.size;
      const int per = (own + kThreads - 1) / kThreads;
      const int first = (int)threadIdx.x * per;
      constexpr int kPer = (kBins + kThreads - 1) / kThreads;
      auto edge = [&](int bin) {  // the weight at a bin's upper edge (times 2^(-1/512), as everywhere)
        const int k = top_grid - 4 * bin;
        return fixed(Weight{s.table[k & 255], min(rw.top - (k >> 8), 63)});
      };
      u64 v[2] = {0, 0};  // logits, estimated weight
      for (int i = 0; i < per && first + i < own; ++i) {
        const int bin = (int)cl.rank * own + first + i;
        uint32_t c = s.hist[bin];
        for (uint32_t r = 1; r < cl.size; ++r) c += cluster_ld(s.hist + bin, cl.rank ^ r);
        s.hist[bin] = c;
        v[0] += c & kCountMask;
        v[1] += bin_estimate(c, edge(bin));
      }
      cl.block_sum(v);
      const u64(*const shares)[kClusterMax] = cl.exchange(v);
      u64 n_all = 0, e_all = 0, share_n[kClusterMax], share_e[kClusterMax];
#pragma unroll
      for (int r = 0; r < kClusterMax; ++r) {
        share_n[r] = r < (int)cl.size ? shares[0][r] : 0;
        share_e[r] = r < (int)cl.size ? shares[1][r] : 0;
        n_all += share_n[r];
        e_all += share_e[r];
      }
      u64 need = (u64)top_k;
      if (!by_weight && n_all <= need) continue;  // the support holds no more
      u64 aim = by_weight ? max(share_of(share, e_all), 1ull) : need;
      // what the bisection below searches: (low, high], `above` already there
      float low = base, high = m;
      u64 above = 0;
      bool found = false;
      float border = -INFINITY;
      for (int attempt = 0; attempt < kTries && !found; ++attempt) {
        // the share, then the bin in it, where the running sum reaches the aim
        int owner = 0;
        u64 n_before = 0, e_before = 0;
#pragma unroll
        for (int r = 0; r + 1 < kClusterMax; ++r)
          if (owner == r && r + 1 < (int)cl.size && (by_weight ? e_before + share_e[r] : n_before + share_n[r]) < aim) {
            n_before += share_n[r];
            e_before += share_e[r];
            owner = r + 1;
          }
        uint32_t word[kPer];
        u64 n_here = 0, e_here = 0, scrap;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          word[i] = i < per && first + i < own ? cluster_ld(s.hist + owner * own + first + i, (uint32_t)owner) : 0;
          n_here += word[i] & kCountMask;
          if (by_weight && word[i]) e_here += bin_estimate(word[i], edge(owner * own + first + i));
        }
        n_before += cl.scan(n_here, &scrap) - n_here;
        if (by_weight) e_before += cl.scan(e_here, &scrap) - e_here;
        if (threadIdx.x == 0) {
          s.found = 0;
          s.bins[0] = kBins;
          s.bins[1] = -1;
          s.count = 0;
        }
        __syncthreads();
        // the last bin in use whose running sum before it is below the aim
        {
          u64 n = n_before, e = e_before;
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (word[i]) {
              if ((by_weight ? e : n) < aim) atomicMax(&s.found, (uint32_t)(owner * own + first + i) + 1);
              n += word[i] & kCountMask;
              if (by_weight) e += bin_estimate(word[i], edge(owner * own + first + i));
            }
        }
        __syncthreads();
        if (s.found == 0) break;  // a second guess beyond the last logit
        const int cross = (int)s.found - 1;
        u64 n = n_before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (owner * own + first + i == cross && i < per) {
            s.before[0] = n;
            s.before[1] = word[i] & kCountMask;
          }
          n += word[i] & kCountMask;
        }
        __syncthreads();
        const u64 n_cross = s.before[0];
        const int in_cross = (int)s.before[1];
        const bool heavy = in_cross > kList;
        // the window: for top-p as many bins on both sides as fit the list
        const u64 margin = by_weight && !heavy ? (u64)(kList - in_cross) / 2 : 0;
        n = n_before;
        u64 e = e_before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int bin = owner * own + first + i;
          if (i < per && first + i < own) {
            if (bin <= cross && n_cross - n <= margin) atomicMin(&s.bins[0], bin);
            if (bin >= cross && n + (word[i] & kCountMask) <= n_cross + in_cross + margin) atomicMax(&s.bins[1], bin);
          }
          n += word[i] & kCountMask;
        }
        __syncthreads();
        const int b0 = margin ? s.bins[0] : cross, b1 = margin ? s.bins[1] : cross;
        if (by_weight) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int bin = owner * own + first + i;
            if (bin == b0 && i < per) s.before[2] = e;
            if (word[i]) e += bin_estimate(word[i], edge(bin));
          }
          __syncthreads();
        }
        // the exact weight above the window and of all, and what is in the window
        u64 sums[3] = {0, 0, 0};
        uint32_t key_min = 0xFFFFFFFFu, key_max = 0;
        sl.template each<kResident>([&](float x, int i) {
          if (x >= base) {
            float off;
            const int b = grid_of(x, &off) >> 2;
            if (by_weight) {
              const u64 w = weight(x);
              sums[1] += w;
              if (b < b0) sums[0] += w;
            }
            if (b >= b0 && b <= b1) {
              if (heavy) {
                key_min = min(key_min, key_of(x));
                key_max = max(key_max, key_of(x));
              } else {
                collect(x, i);
              }
            }
          }
        });
        if (heavy) {
          key_max = cl.max(key_max);
          __syncthreads();
          key_min = ~cl.max(~key_min);
          __syncthreads();
        } else {
          __syncthreads();
          if (threadIdx.x == 0) sums[2] = (u64)s.count;
        }
        u64 mine[3] = {sums[0], sums[1], sums[2]};
        const u64(*const all)[kClusterMax] = cl.sum(mine);
        above = by_weight ? mine[0] : n_cross;
        if (by_weight) need = max(share_of(share, mine[1]), 1ull);
        if (heavy) {
          // in the bin or beside it?  (low, high] covers the bin where it is inside
          u64 in_bin[1] = {0};
          low = key_float(key_min);
          high = key_float(key_max);
          sl.template each<kResident>([&](float x, int) {
            if (x >= low && x <= high) in_bin[0] += by_weight ? weight(x) : 1;
          });
          __syncthreads();
          cl.sum(in_bin);
          if (above >= need || above + in_bin[0] < need) {
            low = base;
            high = m;
            above = 0;
          }
          break;
        }
        const int n_list = (int)mine[2];
        bring(all[2], n_list);
        sort_list(s.list, s.sorted, n_list);
        const u64 c = (int)threadIdx.x < n_list ? s.sorted[threadIdx.x] : 0;
        const u64 w = !c ? 0 : (by_weight ? weight(key_float((uint32_t)(c >> 32))) : 1);
        u64 in_list;
        const u64 upto = above + cl.scan(w, &in_list);
        if (above < need && need <= above + in_list) {
          if (upto >= need && upto - w < need) s.found = (uint32_t)(c >> 32);
          __syncthreads();
          border = key_float(s.found);
          found = true;
        } else {
          // the exact sums say by how much the estimate was off
          const long long next = (long long)s.before[2] + (long long)(need - above);
          aim = next < 1 ? 1 : (u64)next;
          low = base;
          high = m;
          above = 0;
          cl.sync();  // nobody reads the candidates any more
        }
      }
      if (!found) {
        // the largest key whose logits, up to `high`, reach what is needed; `low` does
        uint32_t from = key_of(low), to = key_of(high);
        while (from < to) {
          const uint32_t mid = from + (to - from) / 2 + 1;
          const float vmid = key_float(mid);
          u64 c[1] = {0};
          sl.template each<kResident>([&](float x, int) {
            if (x >= vmid && x <= high) c[0] += by_weight ? weight(x) : 1;
          });
          __syncthreads();
          cl.sum(c);
          if (above + c[0] >= need)
            from = mid;
          else
            to = mid - 1;
        }
        border = key_float(from);
      }
      base = fmaxf(base, border);
      theta = fmaxf(theta, border);
    }

    // ---- the draw, in the order of the vocabulary
    u64 mine = 0;
    sl.template each<kResident>([&](float x, int) {
      if (x >= theta) mine += weight(x);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
    __syncthreads();
    u64 sums[1] = {lane == 0 ? mine : 0};
    const u64(*const all)[kClusterMax] = cl.sum(sums);
    total = sums[0];
    const u64 target = min(__umul64hi(chance, total), total - 1);
    u64 before = 0;
    for (uint32_t r = 0; r < cl.rank; ++r) before += all[0][r];
    for (int w = 0; w < warp; ++w) before += s.warp_sum[0][w];
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
          w[i] = x[i] >= theta ? weight(x[i]) : 0;
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
          if (probs && greedy)
            for (uint32_t r = 0; r < cl.size; ++r) cluster_st(cluster_map(&s.token, r), (uint32_t)token);
        }
        run += __shfl_sync(0xFFFFFFFFu, incl, 31);
        if (run > target) break;
      }
    }
  }
  cl.sync();  // the token is known; no CTA reads another's shared memory any more
  if (!probs) return;
  if (greedy) {
    for (int i = threadIdx.x; i < sl.n; i += kThreads) probs[i] = lo + i == s.token ? 1.f : 0.f;
    return;
  }
  if (threadIdx.x == 0) s.delta[0] = (float)(1.0 / (double)total);
  __syncthreads();
  const float inv = s.delta[0];
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
constexpr size_t kStageTwo = 86 * 1024;   // two CTAs of an SM keep their slices
constexpr size_t kStageOne = 196 * 1024;  // one CTA does

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
  if (!temperature && !(temperature_all <= kHottest)) return SV_ERR_SHAPE;
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
  a.ln_min_p_all = !min_p && min_p_all > 0.f && min_p_all < 1.f ? log((double)min_p_all) : 0.0;
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
