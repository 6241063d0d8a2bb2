// sampling.cuh -- drawing a token from one row of logits, by a thread-block cluster whose CTAs take a slice each.
//
// Mathematics.  With w_v = exp((x_v - m) / T) the filters min-p, top-k and top-p each keep a prefix of the candidates
// in the order (x descending, id ascending), so the set kept is described by one cut (cut_x, cut_id): v is kept iff
// x_v > cut_x, or x_v == cut_x and v <= cut_id.  min-p is a cut at a value.  The top-k cut is the element of a given
// rank, the top-p cut the element at which the running weight reaches a given mass.  Neither needs a sort of the row:
// a histogram over m - x (any monotone function of x will do) names the bin that the border lies in.  When the elements
// in that bin and above it fit a list, every CTA gets them and finishes the draw by itself; otherwise the bin's
// elements alone are listed to find the cut, and only if even those are too many (heavy ties) does cut_by_key() narrow
// an interval of keys down to one value and its ids.  A small top-k needs no histogram of the row: a few of a CTA's
// thread maxima give a floor that few of its elements pass, and the list of all that do shows whether that was enough.
// The draw is an inverse CDF over the kept weights in id order.
//
// Weights become 64-bit integers (multiples of 2^-f of the largest): integer sums are exact, so neither atomics nor the
// split over CTAs changes a result.
//
// What bounds it: with many rows the instructions of a pass over the weights (512 bf16 rows of 151936 entries without
// filters, 156 us: 48 instructions an element, about 32 of them the weight and 10 float64; 75 % of the issue slots used
// while an SM is active, the float64 pipe 35 % busy).  With few rows, latency: a barrier of the cluster takes 0.5 to 1
// us, and a draw passes three (small top-k), seven (top-p alone) or about a dozen (large top-k with top-p) of them.
#pragma once

#include <cooperative_groups.h>

#include <climits>

#include "jf_device.cuh"
#include "jf_math.cuh"
#include "serving_internal.h"

namespace jf {
namespace smp {

#ifdef JF_DEBUG
// Debug build only: while nonzero, a CTA announces the copy of its slice to its barrier but does not issue it, so that
// the wait for it runs out (set by jf_debug_hold; one in each translation unit).
static __device__ int g_hold;
#endif

namespace cg = cooperative_groups;
using u64 = unsigned long long;

// 2^(j/128) for the weights' exponentials (each translation unit keeps its own copy)
static __device__ const double g_exp2_frac128[128] = JF_EXP2_FRAC128;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBinBits = 11;
constexpr int kBins = 1 << kBinBits;
constexpr int kGroupBins = kBins / 32;  // bins in 32 groups: a warp finds the group, then the bin in it, two a lane
static_assert(kGroupBins == 64, "two bins a lane");
constexpr int kList = 1024;          // elements that a list holds: at most two per thread
constexpr int kExpTab = 32, kExpCopies = 16;
constexpr int kSmall = 64;           // lists up to this length: eight threads an element
constexpr int kCounted = kThreads;   // lists up to this length are ordered by counting instead of sorting
constexpr float kBinRange = 32.f;    // the histogram spans at most e^-32 of the largest weight

struct RowParams {
  double t, inv_t;    // T, 1 / T (1 when greedy)
  double ln_min_p_t;  // T ln(min_p), -inf when off
  double top_p;
  float u;
  int top_k;
  bool greedy, ok;
};

struct Smem {
  uint32_t lo[kBins], hi[kBins];       // histogram: elements in lo, or their weight in both words
  double tab[kExpTab * kExpCopies];    // 2^(j / 32), a copy for each lane of a half-warp: no bank conflicts
  u64 mine[kList];                     // scratch of a list's size
  alignas(16) u64 list[kList];         // (ordered key of x, ~id): greater = earlier in the order
  u64 group[kMaxCluster][32];          // every CTA's sums of its groups of bins, written by them
  uint2 part[kMaxCluster];             // every CTA's share of the list, and the floor of its elements
  u64 xch[2][kMaxCluster][2];  // one pair of words per CTA of the cluster, double-buffered
  u64 res[4];                  // what the CTA that holds a border found (written by it into every CTA)
  u64 wsum[2][kWarps];
  float wmax[kWarps], wmin[kWarps];
  uint4 edge[2];  // first and last granule of a slice that is read from global memory
  u64 target, before;  // the border sought, and what lies before the bin that it was found in
  uint32_t bin, border, fill;
  int whole;            // whether a list will hold the bin and all before it
  RowParams rp;
  uint64_t bar;
};

// shared memory of one CTA: Smem, then the slice of the row
constexpr size_t kSliceOff = (sizeof(Smem) + 127) & ~size_t(127);

// what the kernels may ask for
constexpr size_t kMaxDynSmem = 210 * 1024;
constexpr int kMinSlice = 1024;  // entries per CTA below which a wider cluster is no use
constexpr size_t kTwoPerSm = 112 * 1024;  // of each of two CTAs on an SM

// entries per CTA: a multiple of 8, so that a 16-byte granule belongs to one CTA when rows are aligned
__host__ __device__ constexpr int slice_len(int vocab, int cluster) {
  return ((vocab + cluster - 1) / cluster + 7) & ~7;
}
__host__ __device__ constexpr size_t slice_bytes(int vocab, int cluster, int esize) {
  return (static_cast<size_t>(slice_len(vocab, cluster)) * esize + 32 + 127) & ~size_t(127);
}

inline int sm_count() {
  static std::atomic<int> counts[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return -1;
  int n = counts[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    counts[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// The widest cluster with which all rows (or sequences) run at once on an SM a CTA, while a slice keeps kMinSlice
// entries.  Clusters of 16 fill most of a GPC and wait for room once there are more than a few (8 walks of 11 steps
// over float32 rows of 151936 entries: 223 us with 16 CTAs each and 133 with 8 under a small top-k, top-p and min-p,
// 236 and 237 under top-p alone; one walk of 6 steps: 62 and 70 us).
inline int widest_cluster(long long rows, int vocab, int sms) {
  int c = 1;
  while (c < kMaxCluster && rows * 2 * c <= (c < 8 ? sms : sms / 2) && slice_len(vocab, c) > kMinSlice) c *= 2;
  return c;
}

// Sets the attributes of a kernel of this file's users the first time it is launched on a device.
template <typename K>
inline cudaError_t prepare_kernel(K kernel, std::atomic<bool> (&done)[kMaxDevices]) {
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynSmem);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

__device__ __forceinline__ uint32_t ord32(float x) {  // a < b iff ord32(a) < ord32(b); -0 counts as +0
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float ord32_value(uint32_t k) { return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k); }

// Reads and checks the parameters of row r and its random number.
__device__ __forceinline__ RowParams read_params(const SampleParams& sp, long long r, float u) {
  const float t = __ldg(sp.temperature + r);
  const int k = sp.top_k != nullptr ? __ldg(sp.top_k + r) : 0;
  const float tp = sp.top_p != nullptr ? __ldg(sp.top_p + r) : 1.f;
  const float mp = sp.min_p != nullptr ? __ldg(sp.min_p + r) : 0.f;
  RowParams p;
  p.greedy = t == 0.f;  // which leaves the other parameters and u out of account
  p.ok = p.greedy || (t > 0.f && !isinf(t) && k >= 0 && tp >= 0.f && tp <= 1.f && mp >= 0.f && mp <= 1.f &&
                      u >= 0.f && u < 1.f);
  p.t = p.greedy ? 1.0 : static_cast<double>(t);
  p.inv_t = 1.0 / p.t;
  p.ln_min_p_t = mp > 0.f ? static_cast<double>(t) * log(static_cast<double>(mp)) : -INFINITY;
  p.top_p = tp;
  p.u = u;
  p.top_k = k;
  return p;
}

template <typename T>
struct Granule;
template <>
struct Granule<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Granule<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_incl_u64(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

struct Drawn {
  int token;      // -1: no candidate
  float logprob;
  bool ok;        // false: a wait ran out in some CTA of the cluster
  bool mine;      // this thread writes the result (in one thread of the cluster)
};

// Descending bitonic sort of the first n2 entries (a power of two, 64 .. kList) of a list by all threads of the CTA.
// Lane l of warp w holds entries 64 w + l and 64 w + 32 + l; steps over 32 or fewer entries are shuffles, a step over
// 64 or more goes through shared memory.
__device__ __forceinline__ void sort_desc(u64* a, int n2) {
  const int tid = threadIdx.x, lane = tid & 31, i0 = 64 * (tid >> 5) + lane;
  const bool on = i0 < n2;  // whole warps
  u64 v0 = on ? a[i0] : 0, v1 = on ? a[i0 + 32] : 0;
  auto near = [&](int k, int j) {  // compare-exchange across j <= 32 entries
    if (j == 32) {
      const bool desc = (i0 & k) == 0;
      if ((v0 < v1) == desc) {
        const u64 t = v0;
        v0 = v1;
        v1 = t;
      }
      return;
    }
    const u64 o0 = __shfl_xor_sync(0xffffffffu, v0, j), o1 = __shfl_xor_sync(0xffffffffu, v1, j);
    const bool first = (lane & j) == 0;
    const bool big0 = ((i0 & k) == 0) == first, big1 = (((i0 + 32) & k) == 0) == first;
    v0 = (v0 > o0) == big0 ? v0 : o0;
    v1 = (v1 > o1) == big1 ? v1 : o1;
  };
  for (int k = 2; k <= n2; k <<= 1) {
    if (k > 64) {
      __syncthreads();
      if (on) {
        a[i0] = v0;
        a[i0 + 32] = v1;
      }
      for (int j = k >> 1; j >= 64; j >>= 1) {
        __syncthreads();
        const int i = ((tid & ~(j - 1)) << 1) | (tid & (j - 1));
        if (i + j < n2) {
          const u64 x = a[i], y = a[i + j];
          if ((x < y) == ((i & k) == 0)) {
            a[i] = y;
            a[i + j] = x;
          }
        }
      }
      __syncthreads();
      if (on) {
        v0 = a[i0];
        v1 = a[i0 + 32];
      }
    }
    if (on)
      for (int j = k > 64 ? 32 : k >> 1; j > 0; j >>= 1) near(k, j);
  }
  __syncthreads();
  if (on) {
    a[i0] = v0;
    a[i0 + 32] = v1;
  }
  __syncthreads();
}

// One CTA's view of the row, whose slice its warps cut into ranges of consecutive ids.  kResident: the slice lies in
// shared memory, brought there once by a bulk copy; otherwise every pass reads it from global memory (from L2 after the
// first).  Every member function is called by all threads of all CTAs of the cluster, in the same order; the decisions
// between them follow from values that every CTA holds alike.
template <typename T, bool kResident>
struct Row {
  static_assert(kThreads >= kList / 2 && kThreads >= 8 * kSmall && kThreads >= kExpTab * kExpCopies, "work per thread");
  static constexpr int kPer = Granule<T>::n;
  Smem& s;
  uint8_t* buf;       // the slice's granules in shared memory
  const uint4* from;  // or in global memory
  int lo, hi;         // its ids
  int rank, C, tid, lane, warp;
  int vocab, fx;
  int grans;    // 16-byte granules of the slice
  int id0;      // token id of the first element of granule 0 (elements outside the slice hold -inf)
  float m, least;  // largest and smallest candidate
  double md, c32, magic;
  float x_zero;  // below it weights round to 0
  float cut_x;   // the set kept so far
  int cut_id;
  float w_x;     // the same for the elements that weigh anything
  int w_id;
  float top;     // this thread's largest element
  int parity = 0;

  __device__ __forceinline__ Row(Smem& smem, uint8_t* slice, int rank_, int c, int vocab_)
      : s(smem), buf(slice), rank(rank_), C(c), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5),
        vocab(vocab_) {
    const int lg = vocab > 1 ? 32 - __clz(vocab - 1) : 0;
    fx = min(48, 62 - lg);
    magic = __hiloint2double((1023 + 52 - fx) << 20, 0);  // 2^(52 - fx)
    if (tid < kExpTab * kExpCopies) s.tab[tid] = g_exp2_frac128[128 / kExpTab * (tid / kExpCopies)];
    if (tid == 0) {
      mbar_init(&s.bar, 1);
      fence_barrier_init();
    }
  }

  // The double 2^(52 - fx) + exp((x - m) / T), whose mantissa holds round(2^fx exp(..)), for x_zero <= x <= m.  With
  // (x - m) / T = (n + r) ln2 / 32, n integer and |r| <= 1/2, exp = 2^(n >> 5) 2^((n & 31) / 32) e^(r ln2 / 32), the
  // last factor by its Taylor series through the fifth power (truncation below 2^-48).  Exactly 2^fx at x = m.
  // A table of 512 entries needs three terms only, but its lookups conflict (6 a clock and SM against 16 here).  There
  // is no branch in it, so that a granule's exponentials run side by side (a branch for one special value cost a
  // factor of three).
  __device__ __forceinline__ u64 weight_bits(float x) const {
    constexpr double kShift = 0x1.8p52;
    constexpr double a1 = 0.69314718055994530942 / kExpTab, a2 = a1 * a1 / 2, a3 = a2 * a1 / 3, a4 = a3 * a1 / 4,
                     a5 = a4 * a1 / 5;
    const double d = static_cast<double>(x) - md;
    const double t = fma(d, c32, kShift);
    const double r = fma(d, c32, kShift - t);
    const double p = fma(fma(fma(fma(fma(a5, r, a4), r, a3), r, a2), r, a1), r, 1.0);
    const int n = __double2loint(t);
    const double e = s.tab[(n & (kExpTab - 1)) * kExpCopies + (lane & (kExpCopies - 1))];
    const double s2 = __hiloint2double(__double2hiint(e) + (n >> 5) * (1 << 20), __double2loint(e));
    return static_cast<u64>(__double_as_longlong(fma(s2, p, magic)));
  }
  __device__ __forceinline__ u64 magic_bits() const { return static_cast<u64>(__double_as_longlong(magic)); }
  __device__ __forceinline__ u64 weight(float x) const { return weight_bits(x) - magic_bits(); }
  __device__ __forceinline__ bool kept(float x, int id) const { return x > cut_x || (x == cut_x && id <= cut_id); }
  __device__ __forceinline__ int id_of(int g, int e) const { return id0 + g * kPer + e; }
  __device__ __forceinline__ uint4 load(int g) const {
    if (kResident) return reinterpret_cast<const uint4*>(buf)[g];
    uint4 v = make_uint4(0, 0, 0, 0);
    if (g > 0 && g < grans - 1) v = __ldcg(from + g);
    return v;
  }
  // What load() gave, or the granule from s.edge: the first and the last of a slice in global memory may hold entries
  // that are not the slice's, or not even the caller's.
  __device__ __forceinline__ void unpack(int g, uint4 v, float (&x)[kPer]) const {
    if (!kResident && (g == 0 || g == grans - 1)) v = s.edge[g == 0 ? 0 : 1];
    Granule<T>::unpack(v, x);
  }
  __device__ __forceinline__ void warp_range(int w, int& g0, int& g1) const {
    const int gw = (grans + kWarps - 1) / kWarps;
    g0 = min(grans, w * gw);
    g1 = min(grans, g0 + gw);
  }
  // f(g, x) for every granule of this warp's range, in the order of the ids over iterations and lanes; kBatch at a
  // time, and those from global memory are loaded while the batch before them is worked on (256 rows of 151936 float32
  // entries, loaded right before their use: no filter 114 us instead of 105, top-p 295 instead of 278).
  template <int kBatch, typename F>
  __device__ __forceinline__ void walk(F f) const {
    int g0, g1;
    warp_range(warp, g0, g1);
    if constexpr (kResident) {
#pragma unroll kBatch
      for (int g = g0 + lane; g < g1; g += 32) {
        float x[kPer];
        unpack(g, load(g), x);
        f(g, x);
      }
      return;
    }
    uint4 nx[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (g0 + lane + i * 32 < g1) nx[i] = load(g0 + lane + i * 32);
#pragma unroll 1
    for (int g = g0 + lane; g < g1; g += kBatch * 32) {
      uint4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        v[i] = nx[i];
        if (g + (i + kBatch) * 32 < g1) nx[i] = load(g + (i + kBatch) * 32);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (g + i * 32 < g1) {
          float x[kPer];
          unpack(g + i * 32, v[i], x);
          f(g + i * 32, x);
        }
    }
  }
  __device__ __forceinline__ void set_cut(float x, int id) {
    cut_x = x;
    cut_id = id;
    w_x = fmaxf(x, x_zero);
    w_id = x >= x_zero ? id : INT_MAX;
  }
  // Takes the elements of a granule that the cut leaves out among those equal to it; the others are told by x >= w_x.
  // false if none is kept and weighs anything.
  __device__ __forceinline__ bool weighty(int g, float (&x)[kPer]) const {
    if (w_id != INT_MAX) {
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (x[e] == w_x && id_of(g, e) > w_id) x[e] = -INFINITY;
    }
    float top_x = fmax3(x[0], x[1], x[2]);
#pragma unroll
    for (int e = 3; e + 1 < kPer; e += 2) top_x = fmax3(top_x, x[e], x[e + 1]);
    return fmaxf(top_x, x[kPer - 1]) >= w_x;
  }
  // The kept weights of granule g (0 for the others); false if there are none.
  __device__ __forceinline__ bool weights(int g, const float (&in)[kPer], u64 (&w)[kPer]) const {
    float x[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      x[e] = in[e];
      w[e] = 0;
    }
    if (!weighty(g, x)) return false;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const u64 v = weight(x[e]);  // unused where the element is not taken
      w[e] = x[e] >= w_x ? v : 0;
    }
    return true;
  }
  // Their sum.
  __device__ __forceinline__ u64 weight_sum(int g, const float (&in)[kPer]) const {
    float x[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = in[e];
    u64 sum = 0;
    if (weighty(g, x)) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const u64 v = weight(x[e]);
        if (x[e] >= w_x) sum += v;
      }
    }
    return sum;
  }

  // Takes this CTA's slice of a row; a resident one starts on its way to shared memory.  The base of the logits is
  // 16-byte aligned, so the granule that the slice starts in belongs to them.
  __device__ __forceinline__ void start(const T* row) {
    const int per = slice_len(vocab, C);
    lo = min(vocab, rank * per);
    hi = min(vocab, lo + per);
    const int head = static_cast<int>(reinterpret_cast<uintptr_t>(row + lo) & 15) / static_cast<int>(sizeof(T));
    id0 = lo - head;
    grans = lo < hi ? (hi - id0 + kPer - 1) / kPer : 0;
    from = reinterpret_cast<const uint4*>(row + id0);
    if (!kResident) {
      if (tid < 2 * kPer && grans > 0) {
        const int id = id0 + (tid < kPer ? 0 : (grans - 1) * kPer) + tid % kPer;
        reinterpret_cast<T*>(&s.edge)[tid] = id >= lo && id < hi ? row[id] : static_cast<T>(-INFINITY);
      }
      return;
    }
    const int full = lo < hi ? (hi - id0) / kPer : 0;
    if (tid == 0) {
      mbar_arrive_expect_tx(&s.bar, full * 16);
      bool issue = full > 0;
#ifdef JF_DEBUG
      issue = issue && *reinterpret_cast<volatile int*>(&g_hold) == 0;
#endif
      if (issue)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                smem_u32(buf)),
            "l"(from), "r"(full * 16), "r"(smem_u32(&s.bar))
            : "memory");
    }
    // the last granule's elements, when the slice ends inside one
    const int id = id0 + full * kPer + tid;
    if (full < grans && tid < kPer)
      reinterpret_cast<T*>(buf)[full * kPer + tid] = id < hi ? row[id] : static_cast<T>(-INFINITY);
  }
  // Waits for it (bounded) and clears what lies before it in its first granule.
  __device__ __forceinline__ bool finish(uint32_t phase) {
    if (!kResident) {
      __syncthreads();
      return true;
    }
    volatile int never = 0;
    const bool ok = mbar_wait(&s.bar, phase, &never);
    if (grans > 0 && tid < lo - id0) reinterpret_cast<T*>(buf)[tid] = static_cast<T>(-INFINITY);
    return __syncthreads_and(ok);
  }

  // Brings this CTA's slice of a row into L2 (whole granules inside the row).
  __device__ __forceinline__ void prefetch(const T* row) const {
    const int per = slice_len(vocab, C);
    const int lo = min(vocab, rank * per), hi = min(vocab, lo + per);
    const uintptr_t a = (reinterpret_cast<uintptr_t>(row + lo) + 15) & ~uintptr_t(15);
    const uintptr_t e = reinterpret_cast<uintptr_t>(row + hi) & ~uintptr_t(15);
    if (a < e)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"(static_cast<uint32_t>(e - a))
                   : "memory");
  }

  // Every CTA's pair of words, in s.xch[result] afterwards; a and b need to be valid in threads 0 .. C-1.
  __device__ __forceinline__ int exchange(u64 a, u64 b) {
    const int p = parity;
    parity ^= 1;
    if (tid < C) {
      u64* dst = cg::this_cluster().map_shared_rank(&s.xch[p][rank][0], tid);
      dst[0] = a;
      dst[1] = b;
    }
    cg::this_cluster().sync();
    return p;
  }

  // The row's largest and smallest candidate; m = -inf if there is none.
  __device__ __forceinline__ bool find_range(bool ok) {
    float mx = -INFINITY, mn = INFINITY;
    walk<4>([&](int, const float(&x)[kPer]) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        mx = fmaxf(mx, x[e]);  // NaN drops out
        mn = fminf(mn, x[e] == -INFINITY ? INFINITY : x[e]);
      }
    });
    top = mx;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    if (lane == 0) {
      s.wmax[warp] = mx;
      s.wmin[warp] = mn;
    }
    __syncthreads();
    mx = s.wmax[lane & (kWarps - 1)];
    mn = s.wmin[lane & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    const int p = exchange(__float_as_uint(mx) | static_cast<u64>(__float_as_uint(mn)) << 32, ok ? 1 : 0);
    bool all = true;
    m = -INFINITY;
    least = INFINITY;
    for (int c = 0; c < C; ++c) {
      const u64 v = s.xch[p][c][0];
      m = fmaxf(m, __uint_as_float(static_cast<uint32_t>(v)));
      least = fminf(least, __uint_as_float(static_cast<uint32_t>(v >> 32)));
      all = all && s.xch[p][c][1] != 0;
    }
    md = static_cast<double>(m);
    return all;
  }

  // Exclusive prefix of (a, b) over the CTA's threads and the CTA's totals.
  __device__ __forceinline__ void block_scan(u64 a, u64 b, u64& ea, u64& eb, u64& ta, u64& tb) {
    const u64 ia = warp_incl_u64(a, lane), ib = warp_incl_u64(b, lane);
    __syncthreads();
    if (lane == 31) {
      s.wsum[0][warp] = ia;
      s.wsum[1][warp] = ib;
    }
    __syncthreads();
    ea = ia - a;
    eb = ib - b;
    ta = tb = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
        ea += ta;
        eb += tb;
      }
      ta += s.wsum[0][w];
      tb += s.wsum[1][w];
    }
  }

  __device__ __forceinline__ void add_mass(int bin, u64 w) {
    const uint32_t add = static_cast<uint32_t>(w), old = atomicAdd(&s.lo[bin], add);
    const uint32_t up = static_cast<uint32_t>(w >> 32) + (old + add < old ? 1u : 0u);
    if (up != 0) atomicAdd(&s.hi[bin], up);
  }
  // The same for a granule, without a branch between its elements (those not taken add 0).
  __device__ __forceinline__ void add_masses(const float (&x)[kPer], const u64 (&w)[kPer]) {
    uint32_t old[kPer], up[kPer], any = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) old[e] = atomicAdd(&s.lo[bin_of(x[e])], static_cast<uint32_t>(w[e]));
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      up[e] = static_cast<uint32_t>((w[e] + old[e]) >> 32);
      any |= up[e];
    }
    if (any != 0) {
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (up[e] != 0) atomicAdd(&s.hi[bin_of(x[e])], up[e]);
    }
  }
  __device__ __forceinline__ void clear_bins() {
    for (int i = tid; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0;
    __syncthreads();
  }

  // Bins in the order of the candidates: bin 0 holds the largest.
  float bin_scale;
  __device__ __forceinline__ int bin_of(float x) const {
    const float d = fminf((m - x) * bin_scale, static_cast<float>(kBins - 1));
    return __float_as_int(d + 12582912.f) & 0x7fffff & (2 * kBins - 1);  // rint(d), by adding 1.5 * 2^23
  }
  __device__ __forceinline__ void set_bins(const RowParams& rp) {
    const float span = fminf(static_cast<float>(kBinRange * rp.t), m - least);
    bin_scale = span > 0.f ? fminf(static_cast<float>(kBins - 1) / span, 1e37f) : 0.f;
  }

  // Fills the histogram with the kept elements and finds the bin that holds element number k (mass false) or at which
  // the running weight reaches the share top_p of the whole (mass true): s.bin, s.target and what lies before the bin.
  // false, with no bin, if there are no more than k elements.
  __device__ __forceinline__ bool find_bin(bool mass, u64 k, double share) {
    clear_bins();
    if (mass) {
      walk<1>([&](int g, const float(&x)[kPer]) {
        u64 w[kPer];
        if (weights(g, x, w)) add_masses(x, w);
      });
    } else {
      walk<4>([&](int g, const float(&x)[kPer]) {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (kept(x[e], id_of(g, e))) atomicAdd(&s.lo[bin_of(x[e])], 1u);
      });
    }
    __syncthreads();
    cg::cluster_group cl = cg::this_cluster();
    // the sums of this CTA's groups of bins go to every CTA
    for (int g = warp; g < 32; g += kWarps) {
      const int b = g * kGroupBins + lane;
      const u64 w = (s.lo[b] | static_cast<u64>(s.hi[b]) << 32) + (s.lo[b + 32] | static_cast<u64>(s.hi[b + 32]) << 32);
      const u64 sum = warp_sum_u64(w);
      if (lane < C) *cl.map_shared_rank(&s.group[rank][g], lane) = sum;
    }
    cl.sync();  // the histograms stay as they are until the next cluster barrier
    if (warp == 0) {
      u64 w = 0;  // lane = group of bins
      for (int c = 0; c < C; ++c) w += s.group[c][lane];
      const u64 iw = warp_incl_u64(w, lane), total = __shfl_sync(0xffffffffu, iw, 31);
      u64 target = k;
      if (mass) {
        target = static_cast<u64>(ceil(share * static_cast<double>(total)));
        target = target < 1 ? 1 : (target > total ? total : target);
      }
      if (target < total || mass) {
        const int grp = __ffs(__ballot_sync(0xffffffffu, iw >= target)) - 1;
        const u64 w0 = __shfl_sync(0xffffffffu, iw - w, grp);
        u64 v[2] = {0, 0};  // lane = two bins of that group
#pragma unroll 8
        for (int c = 0; c < C; ++c) {
          const uint2 lo2 = *reinterpret_cast<const uint2*>(cl.map_shared_rank(&s.lo[grp * kGroupBins + 2 * lane], c));
          const uint2 hi2 = *reinterpret_cast<const uint2*>(cl.map_shared_rank(&s.hi[grp * kGroupBins + 2 * lane], c));
          v[0] += lo2.x | static_cast<u64>(hi2.x) << 32;
          v[1] += lo2.y | static_cast<u64>(hi2.y) << 32;
        }
        const u64 upto = w0 + warp_incl_u64(v[0] + v[1], lane);
        const int at = __ffs(__ballot_sync(0xffffffffu, upto >= target)) - 1;
        if (lane == at) {
          const bool second = upto - v[1] < target;
          const int bin = grp * kGroupBins + 2 * lane + (second ? 1 : 0);
          const u64 in_bin = v[second ? 1 : 0], before = upto - v[1] - (second ? 0 : v[0]);
          s.bin = bin;
          s.before = before;
          // a list of all elements up to the bin is worth a try if their number, or from the mass that of the bin and
          // some bins before it, is not too large
          const float x = fminf(m, m - static_cast<float>(bin) / bin_scale);
          const u64 w = mass ? (x >= x_zero ? weight(x) : 1) : 1;
          s.whole = mass ? in_bin <= w * (kList / 16) : before + in_bin <= kList;
        }
      } else if (lane == 0) {
        s.bin = kBins;
      }
      if (lane == 0) s.target = target;
    }
    __syncthreads();
    return s.bin < kBins;
  }

  // A value below every value of the bin, and one above every value, each by less than two bins.
  __device__ __forceinline__ float below_bin(int bin) const {
    return bin_scale > 0.f && bin < kBins - 1 ? m - static_cast<float>(bin + 2) / bin_scale : -INFINITY;
  }
  __device__ __forceinline__ float above_bin(int bin) const {
    return bin_scale > 0.f && bin > 2 ? m - static_cast<float>(bin - 2) / bin_scale : INFINITY;
  }
  // Writes this CTA's kept elements from `floor` on to s.mine, with only >= 0 those of that bin alone; s.fill counts
  // them, or exceeds kList.  Few are: most granules end at the comparison with the two bounds.
  __device__ __forceinline__ void gather(float floor, int only) {
    __syncthreads();
    if (tid == 0) s.fill = 0;
    __syncthreads();
    const float ceiling = only >= 0 ? above_bin(only) : INFINITY;
    walk<2>([&](int g, const float(&x)[kPer]) {
      uint32_t hits = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) hits |= x[e] >= floor && x[e] <= ceiling ? 1u << e : 0u;
      if (hits == 0 || *static_cast<volatile uint32_t*>(&s.fill) > kList) return;
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (!kept(x[e], id_of(g, e)) || (only >= 0 && bin_of(x[e]) != only)) hits &= ~(1u << e);
      if (hits == 0) return;
      uint32_t at = atomicAdd(&s.fill, static_cast<uint32_t>(__popc(hits)));
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (hits >> e & 1) {
          if (at < kList) s.mine[at] = static_cast<u64>(ord32(x[e])) << 32 | static_cast<uint32_t>(~id_of(g, e));
          ++at;
        }
    });
    __syncthreads();
  }
  // Copies this CTA's s.fill entries to place `at` of every CTA's list.
  __device__ __forceinline__ void put(int at) {
    const int lg = 31 - __clz(C);  // C is a power of two
    for (int i = tid; i < static_cast<int>(s.fill) << lg; i += kThreads)
      *cg::this_cluster().map_shared_rank(&s.list[at + (i >> lg)], i & (C - 1)) = s.mine[i >> lg];
  }
  __device__ __forceinline__ void order(int n) {
    if (n <= kSmall) {  // eight threads count an element's rank
      const int i = tid / 8;
      const u64 v = i < n ? s.list[i] : 0;
      int rank_of = 0;
      for (int j = tid % 8; j < n; j += 8) rank_of += s.list[j] > v;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) rank_of += __shfl_xor_sync(0xffffffffu, rank_of, o);
      __syncthreads();
      if (i < n && tid % 8 == 0) s.list[rank_of] = v;
      __syncthreads();
      return;
    }
    if (n <= kCounted) {  // a thread counts an element's, two entries a load (the one behind the last is 0)
      if (tid == 0 && (n & 1)) s.list[n] = 0;
      __syncthreads();
      const u64 v = tid < n ? s.list[tid] : ~0ull;
      int rank_of = 0;
      if (tid < ((n + 31) & ~31)) {
        const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(s.list);
#pragma unroll 4
        for (int j = 0; j < (n + 1) / 2; ++j) rank_of += (pairs[j].x > v) + (pairs[j].y > v);
      }
      __syncthreads();
      if (tid < n) s.list[rank_of] = v;
      __syncthreads();
      return;
    }
    int n2 = 64;
    while (n2 < n) n2 *= 2;
    if (tid < n2 - n) s.list[n + tid] = 0;  // n2 - n < kThreads
    __syncthreads();
    sort_desc(s.list, n2);
  }

  // Lists what is kept up to the bin found, or that bin alone (whole becomes false), in every CTA and in order; the
  // number, 0 if even that is more than a list holds.
  __device__ __forceinline__ int list_bin(bool& whole) {
    u64 n = 0;
#pragma unroll 1
    for (int alone = s.whole ? 0 : 1; alone < 2; ++alone) {
      gather(below_bin(static_cast<int>(s.bin)), alone ? static_cast<int>(s.bin) : -1);
      const int p = exchange(s.fill, 0);
      u64 base = 0;
      n = 0;
      for (int c = 0; c < C; ++c) {
        if (c < rank) base += s.xch[p][c][0];
        n += s.xch[p][c][0];
      }
      whole = alone == 0;
      if (n > kList) continue;
      put(static_cast<int>(base));
      cg::this_cluster().sync();
      order(static_cast<int>(n));
      return static_cast<int>(n);
    }
    return 0;
  }

  // Lists a superset of the k largest kept elements in every CTA, in order: each CTA's elements from a floor on, which
  // is the bin of the `local`-th largest of its thread maxima.  Elements missing lie below their CTA's floor, so the k
  // largest are known if the k-th of the list reaches the highest floor; the number, or 0 if that does not work out (k
  // too large, uneven CTAs, ties).
  __device__ __forceinline__ int list_largest(int k) {
    const int room = kList / C, local = min(k, 3 * k / C + 8);
    if (local > room / 2 || local > kThreads / 2) return 0;
    clear_bins();
    if (kept(top, -1)) atomicAdd(&s.lo[bin_of(top)], 1u);
    __syncthreads();
    if (warp == 0) {
      uint32_t n = 0;  // lane = group of bins
      for (int i = 0; i < kGroupBins; ++i) n += s.lo[lane * kGroupBins + ((i + lane) & (kGroupBins - 1))];
      uint32_t in = static_cast<uint32_t>(warp_incl_u64(n, lane));
      const uint32_t hit = __ballot_sync(0xffffffffu, in >= static_cast<uint32_t>(local));
      if (hit != 0) {
        const int grp = __ffs(hit) - 1;
        const uint32_t n0 = __shfl_sync(0xffffffffu, in - n, grp);
        const uint2 two = *reinterpret_cast<const uint2*>(&s.lo[grp * kGroupBins + 2 * lane]);
        in = n0 + static_cast<uint32_t>(warp_incl_u64(two.x + two.y, lane));
        const int at = __ffs(__ballot_sync(0xffffffffu, in >= static_cast<uint32_t>(local))) - 1;
        if (lane == at) s.bin = grp * kGroupBins + 2 * lane + (in - two.y < static_cast<uint32_t>(local) ? 1 : 0);
      } else if (lane == 0) {
        s.bin = kBins - 1;  // fewer threads than that have a candidate: all elements
      }
    }
    __syncthreads();
    const float floor = below_bin(static_cast<int>(s.bin));
    gather(floor, -1);
    if (tid < C) *cg::this_cluster().map_shared_rank(&s.part[rank], tid) = make_uint2(s.fill, __float_as_uint(floor));
    if (s.fill <= static_cast<uint32_t>(room)) put(rank * room);
    cg::this_cluster().sync();
    // the parts move together; what lies behind the last is cleared
    int n = 0, most = 0;
    float highest = -INFINITY;
    for (int c = 0; c < C; ++c) {
      n += s.part[c].x;
      most = max(most, static_cast<int>(s.part[c].x));
      highest = fmaxf(highest, __uint_as_float(s.part[c].y));
    }
    if (most > room) return 0;
    u64 v[kList / kThreads];
    int to[kList / kThreads];
#pragma unroll
    for (int i = 0; i < kList / kThreads; ++i) {
      const int from = tid + i * kThreads, c = from / room, at = from % room;
      to[i] = -1;
      if (at < static_cast<int>(s.part[c].x)) {
        v[i] = s.list[from];
        to[i] = at;
        for (int b = 0; b < c; ++b) to[i] += s.part[b].x;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kList / kThreads; ++i)
      if (to[i] >= 0) s.list[to[i]] = v[i];
    __syncthreads();
    order(n);
    const bool known = n >= k ? list_x(k - 1) >= highest : highest == -INFINITY;
    if (!known) {
      cg::this_cluster().sync();  // the list is not written again before every CTA has read it
      return 0;
    }
    return n;
  }
  __device__ __forceinline__ float list_x(int i) const { return ord32_value(static_cast<uint32_t>(s.list[i] >> 32)); }
  __device__ __forceinline__ int list_id(int i) const { return static_cast<int>(~static_cast<uint32_t>(s.list[i])); }
  __device__ __forceinline__ u64 list_weight(int i) const {
    const float x = list_x(i);
    return x >= x_zero ? weight(x) : 0;
  }

  // Index of the first of the list's n elements at which the running weight reaches `target`, which it does.
  __device__ __forceinline__ int list_border(int n, u64 target) {
    const u64 a = 2 * tid < n ? list_weight(2 * tid) : 0, b = 2 * tid + 1 < n ? list_weight(2 * tid + 1) : 0;
    u64 before, e2, total, t2;
    block_scan(a + b, 0, before, e2, total, t2);
    if (before < target && target <= before + a) s.border = 2 * tid;
    else if (before + a < target && target <= before + a + b) s.border = 2 * tid + 1;
    __syncthreads();
    return static_cast<int>(s.border);
  }
  __device__ __forceinline__ u64 list_mass(int n) {
    const u64 a = 2 * tid < n ? list_weight(2 * tid) : 0, b = 2 * tid + 1 < n ? list_weight(2 * tid + 1) : 0;
    u64 e1, e2, total, t2;
    block_scan(a + b, 0, e1, e2, total, t2);
    return total;
  }

  // The draw among the first n elements of the list: the first, by id, whose running weight exceeds u times all.
  __device__ __forceinline__ void draw_from_list(int n, float u, Drawn& d) {
    u64 total;
    if (n <= kSmall) {  // eight threads sum the weights of the ids up to an element's
      const int i = tid / 8;
      if (tid < n) s.mine[tid] = list_weight(tid);
      __syncthreads();
      const uint32_t id = i < n ? static_cast<uint32_t>(list_id(i)) : 0;
      u64 upto = 0, all = 0;
      for (int j = tid % 8; j < n; j += 8) {
        const u64 w = s.mine[j];
        all += w;
        if (static_cast<uint32_t>(list_id(j)) <= id) upto += w;
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        upto += __shfl_xor_sync(0xffffffffu, upto, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
      }
      total = all;
      const u64 t = static_cast<u64>(static_cast<double>(u) * static_cast<double>(total));
      if (i < n && tid % 8 == 0 && upto > t && upto - s.mine[i] <= t) {
        s.res[0] = id;
        s.res[1] = __float_as_uint(list_x(i));
      }
    } else {
      int n2 = 64;
      while (n2 < n) n2 *= 2;
#pragma unroll
      for (int i = 0; i < kList / kThreads; ++i) {  // (~id, ordered key): descending = ascending ids
        const int at = tid + i * kThreads;
        if (at < n2) s.mine[at] = at < n ? s.list[at] << 32 | s.list[at] >> 32 : 0;
      }
      __syncthreads();
      sort_desc(s.mine, n2);
      float x[2];
      u64 w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = 2 * tid + i;
        x[i] = at < n ? ord32_value(static_cast<uint32_t>(s.mine[at])) : -INFINITY;
        w[i] = at < n && x[i] >= x_zero ? weight(x[i]) : 0;
      }
      u64 before, e2, t2;
      block_scan(w[0] + w[1], 0, before, e2, total, t2);
      const u64 t = static_cast<u64>(static_cast<double>(u) * static_cast<double>(total));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (before <= t && t < before + w[i]) {
          s.res[0] = static_cast<uint32_t>(~static_cast<uint32_t>(s.mine[2 * tid + i] >> 32));
          s.res[1] = __float_as_uint(x[i]);
        }
        before += w[i];
      }
    }
    __syncthreads();
    d.token = static_cast<int>(s.res[0]);
    d.logprob = log_prob(__uint_as_float(static_cast<uint32_t>(s.res[1])), total);
    d.mine = rank == 0 && tid == 0;
  }
  __device__ __forceinline__ float log_prob(float x, u64 total) const {
    const double y = (static_cast<double>(x) - md) * (c32 * (0.69314718055994530942 / kExpTab));
    // the weight kept, in units of the largest: at least 1, so that no result is above 0
    const double kept_weight = static_cast<double>(total) * __hiloint2double((1023 - fx) << 20, 0);
    return static_cast<float>(y - log(kept_weight));
  }

  // Narrows the kept set to end at its element number `k` (mass false), or at the element where the running weight
  // reaches `target` (mass true), whatever the values: an interval of keys is narrowed by histograms to one key.  The
  // set is known to hold that much.
  __device__ __forceinline__ void cut_by_key(bool mass, u64 target) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();  // no CTA reads the last histogram any more
    uint32_t base = ord32(m);
    int bits = 32;  // the interval is (base - 2^bits, base]
    while (bits > 0) {
      const int shift = bits > kBinBits ? bits - kBinBits : 0;
      clear_bins();
      walk<2>([&](int g, const float(&x)[kPer]) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (!kept(x[e], id_of(g, e))) continue;
          const uint32_t d = base - ord32(x[e]);  // wraps for keys above the interval
          if (bits < 32 && (d >> bits) != 0) continue;
          if (!mass) atomicAdd(&s.lo[d >> shift], 1u);
          else if (x[e] >= x_zero) add_mass(d >> shift, weight(x[e]));
        }
      });
      cl.sync();  // every CTA's histogram is complete
      // this CTA sums its share of the bins over the cluster: consecutive bins per thread, in order
      const int seg = kBins / C, b0 = rank * seg;
      const int per = (seg + kThreads - 1) / kThreads;
      const int t0 = tid * per;
      u64 sum = 0;
      u64 v[kBins / kThreads];
#pragma unroll
      for (int i = 0; i < kBins / kThreads; ++i) {
        v[i] = 0;
        if (i < per && t0 + i < seg) {
          for (int c = 0; c < C; ++c) {
            v[i] += *cl.map_shared_rank(&s.lo[b0 + t0 + i], c);
            v[i] += static_cast<u64>(*cl.map_shared_rank(&s.hi[b0 + t0 + i], c)) << 32;
          }
          sum += v[i];
        }
      }
      u64 excl, e2, total, t2;
      block_scan(sum, 0, excl, e2, total, t2);
      const int p = exchange(total, 0);
      u64 run = excl;
      for (int c = 0; c < rank; ++c) run += s.xch[p][c][0];
#pragma unroll
      for (int i = 0; i < kBins / kThreads; ++i) {
        if (run < target && target <= run + v[i]) {  // exactly one thread of the cluster
          for (int c = 0; c < C; ++c) {
            u64* r = cl.map_shared_rank(&s.res[0], c);
            r[0] = b0 + t0 + i;
            r[1] = run;
          }
        }
        run += v[i];
      }
      cl.sync();
      base -= static_cast<uint32_t>(s.res[0]) << shift;
      target -= s.res[1];
      bits = shift;
    }
    // the interval is one key: the elements equal to it, in id order
    const float v = ord32_value(base);
    const u64 w1 = mass ? weight(v) : 1;
    const u64 nth = (target + w1 - 1) / w1;
    u64 total;
    float at;
    int id;
    find_equal(v, nth - 1, total, id, at);
    set_cut(v, id);
  }

  // The lowest id at which the running sum of f, in id order, exceeds t, and its value; t is `fixed` if share < 0, else
  // floor(share * total).  f(g, x, w) gives the terms of granule g, sum_of(g, x) their sum.  kAll: every thread of the
  // cluster gets the result; otherwise the thread that returns true does, and all get the total.
  template <bool kAll, typename F, typename S>
  __device__ __forceinline__ bool find_id(u64 fixed, double share, F f, S sum_of, u64& total, int& id, float& at) {
    u64 sum = 0;
    walk<1>([&](int g, const float(&x)[kPer]) { sum += sum_of(g, x); });
    sum = warp_sum_u64(sum);
    __syncthreads();
    if (lane == 0) s.wsum[0][warp] = sum;
    __syncthreads();
    u64 mine = 0;
    for (int w = 0; w < kWarps; ++w) mine += s.wsum[0][w];
    const int p = exchange(mine, 0);
    u64 before = 0;
    total = 0;
    for (int c = 0; c < C; ++c) {
      if (c < rank) before += s.xch[p][c][0];
      total += s.xch[p][c][0];
    }
    const u64 t = share < 0 ? fixed : static_cast<u64>(share * static_cast<double>(total));
    bool found = false;
    if (before <= t && t < before + mine) {  // one CTA of the cluster
      // the warp's range that holds it; one of more than 8 steps is split among the CTA's warps once more, so that the
      // warp that walks it has few left (256 rows of 151936 entries, no filter: 114 us, without the split 146 us)
      int owner = 0, g0, g1;
      for (; owner < kWarps - 1 && before + s.wsum[0][owner] <= t; ++owner) before += s.wsum[0][owner];
      warp_range(owner, g0, g1);
      if (g1 - g0 > 8 * 32) {
        const int part = (g1 - g0 + kWarps - 1) / kWarps, a = min(g1, g0 + warp * part), b = min(g1, a + part);
        u64 sub = 0;
        for (int g = a + lane; g < b; g += 32) {
          float x[kPer];
          unpack(g, load(g), x);
          sub += sum_of(g, x);
        }
        sub = warp_sum_u64(sub);
        if (lane == 0) s.wsum[1][warp] = sub;
        __syncthreads();
        for (owner = 0; owner < kWarps - 1 && before + s.wsum[1][owner] <= t; ++owner) before += s.wsum[1][owner];
        g0 = min(g1, g0 + owner * part);
        g1 = min(g1, g0 + part);
      }
      u64 run = before;
      if (warp != owner) g1 = g0;
      for (int gb = g0; gb < g1; gb += 32) {
        const int g = gb + lane;
        float x[kPer];
        u64 w[kPer], mysum = 0;
        if (g < g1) {
          unpack(g, load(g), x);
          f(g, x, w);
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (g >= g1) w[e] = 0;
          mysum += w[e];
        }
        const u64 incl = run + warp_incl_u64(mysum, lane);
        const uint32_t hit = __ballot_sync(0xffffffffu, incl > t);
        if (hit != 0) {
          if (lane == __ffs(hit) - 1) {
            u64 r = incl - mysum;
            found = true;
            bool done = false;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              r += w[e];
              if (!done && r > t) {
                done = true;
                id = id_of(g, e);
                at = x[e];
              }
            }
            if (kAll)
              for (int c = 0; c < C; ++c) {
                u64* dst = cg::this_cluster().map_shared_rank(&s.res[2], c);
                dst[0] = static_cast<u64>(id);
                dst[1] = __float_as_uint(at);
              }
          }
          break;
        }
        run = __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (kAll) {
      cg::this_cluster().sync();
      id = static_cast<int>(s.res[2]);
      at = __uint_as_float(static_cast<uint32_t>(s.res[3]));
    }
    return found;
  }

  // Number t + 1, in id order, of the kept elements that equal v; their number is the total.
  __device__ __forceinline__ bool find_equal(float v, u64 t, u64& total, int& id, float& at) {
    auto terms = [&](int g, const float(&x)[kPer], u64(&w)[kPer]) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) w[e] = x[e] == v && kept(x[e], id_of(g, e)) ? 1 : 0;
    };
    auto sum_of = [&](int g, const float(&x)[kPer]) {
      u64 w[kPer], sum = 0;
      terms(g, x, w);
#pragma unroll
      for (int e = 0; e < kPer; ++e) sum += w[e];
      return sum;
    };
    return find_id<true>(t, -1.0, terms, sum_of, total, id, at);
  }

  // The whole draw, after start() and with the row's parameters in s.rp.  kAll: the result is wanted in every thread;
  // otherwise in the one whose result says so (and CTAs may return from here while others still work on their own).
  template <bool kAll>
  __device__ __forceinline__ Drawn draw(uint32_t phase) {
    Drawn d{-1, -INFINITY, true, rank == 0 && tid == 0};
    d.ok = find_range(finish(phase));
    const RowParams& rp = s.rp;
    const float u = rp.u;
    if (!d.ok || !rp.ok || m == -INFINITY) return d;
    cut_id = INT_MAX;
    u64 total;
    if (rp.greedy || m == INFINITY) {
      // the candidates that attain the maximum: the first of them or, for +inf, an equal share each
      cut_x = m;
      u64 n = 1, t = 0;
      float at;
#pragma unroll 1
      for (int round = rp.greedy ? 1 : 0; round < 2; ++round) {
        find_equal(m, t, total, d.token, at);
        if (round == 1) break;
        n = rp.top_k > 0 && rp.top_k < total ? rp.top_k : total;
        if (rp.top_p < 1.0) n = max(1ull, static_cast<u64>(ceil(rp.top_p * static_cast<double>(n))));
        t = static_cast<u64>(static_cast<double>(u) * static_cast<double>(n));
      }
      d.logprob = n == 1 ? 0.f : static_cast<float>(-log(static_cast<double>(n)));
      return d;
    }
    c32 = rp.inv_t * (kExpTab / 0.69314718055994530942);
    // Rounded up: a float32 logit is at or above it exactly when it is at or above the bound itself.  Rounded down, the
    // step below a large m could lie hundreds of T under it, where weight_bits() has no exponent left.
    x_zero = __double2float_ru(md - (fx + 2) * 0.69314718055994530942 * rp.t);
    set_cut(fmaxf(__double2float_ru(md + rp.ln_min_p_t), -3.402823466e38f), INT_MAX);
    set_bins(rp);
    // top-k by the count, then top-p by the weight; a list that holds all that is kept ends the draw
    const bool by_k = rp.top_k > 0 && rp.top_k < vocab, by_p = rp.top_p < 1.0;
#pragma unroll 1
    for (int pass = by_k ? 0 : 1; pass < (by_p ? 2 : 1); ++pass) {
      const bool mass = pass == 1;
      bool whole = true;
      u64 target = rp.top_k, before = 0;
      int n = mass ? 0 : list_largest(rp.top_k);
      if (n == 0) {
        if (mass && by_k) cg::this_cluster().sync();  // no CTA reads the last histogram or its groups any more
        if (!find_bin(mass, rp.top_k, rp.top_p)) continue;
        target = s.target;
        before = s.before;
        n = list_bin(whole);
      }
      if (n > 0 && whole) {
        if (!kAll && rank != 0) return d;
        if (!mass) {
          n = min(n, rp.top_k);
          if (by_p) {
            const u64 all = list_mass(n);
            target = max(1ull, static_cast<u64>(ceil(rp.top_p * static_cast<double>(all))));
            target = min(target, all);
          }
        }
        if (by_p) n = 1 + list_border(n, target);
        draw_from_list(n, u, d);
        return d;
      }
      if (n > 0) {
        const int at = mass ? list_border(n, target - before) : static_cast<int>(target - before) - 1;
        set_cut(list_x(at), list_id(at));
        __syncthreads();
      } else {
        cut_by_key(mass, target);
      }
    }
    const bool found = find_id<kAll>(
        0, u, [&](int g, const float(&x)[kPer], u64(&w)[kPer]) { weights(g, x, w); },
        [&](int g, const float(&x)[kPer]) { return weight_sum(g, x); }, total, d.token, d.logprob);
    if (!kAll) d.mine = found;
    d.logprob = log_prob(d.logprob, total);
    return d;
  }
};

}  // namespace smp
}  // namespace jf
