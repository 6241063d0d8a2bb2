// sampling.cuh -- drawing a token from one row of logits that lies in the shared memory of a thread-block cluster.
//
// Mathematics.  With w_v = exp((x_v - m) / T) the filters min-p, top-k and top-p each keep a prefix of the candidates in
// the order (x descending, id ascending), so the set kept is described by one cut (cut_x, cut_id): v is kept iff
// x_v > cut_x, or x_v == cut_x and v <= cut_id.  min-p is a cut at a value.  The top-k cut is the element of a given
// rank, the top-p cut the element at which the running weight reaches a given mass.  Neither needs a sort of the row: a
// histogram over m - x (any monotone function of x will do) names the bin that the border lies in.  When no more than
// kList elements lie in that bin or above it, every CTA gets a list of them and finishes the draw by itself; otherwise
// the bin's elements alone are listed to find the cut, and only if even those are too many (heavy ties) does cut_by_key()
// narrow an interval of keys down to one value and its ids.  A small top-k needs no histogram of the row: the k-th
// largest of a CTA's thread maxima bounds the CTA's k-th largest element from below, and few elements pass that bound.
// The draw is an inverse CDF over the kept weights in id order.
//
// Weights become 64-bit integers (multiples of 2^-f of the largest): integer sums are exact, so neither atomics nor the
// split over CTAs changes a result.
#pragma once

#include <cooperative_groups.h>

#include <climits>

#include "jf_device.cuh"
#include "jf_math.cuh"
#include "serving_internal.h"

namespace jf {
namespace smp {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

// 2^(j/128) for the weights' exponentials (each translation unit keeps its own copy)
static __device__ const double g_exp2_frac128[128] = JF_EXP2_FRAC128;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBinBits = 10;
constexpr int kBins = 1 << kBinBits;
constexpr int kGroups = kBins / 32;  // bins in groups of 32: a warp finds the group, then the bin in it
constexpr int kList = 1024;          // elements that a list holds: two per thread
constexpr int kExpTab = 32, kExpCopies = 16;
constexpr int kSmall = 64;           // lists up to this length are ordered by counting instead of sorting
constexpr float kBinRange = 32.f;    // the histogram spans at most e^-32 of the largest weight

struct Smem {
  uint32_t lo[kBins], hi[kBins];       // histogram: elements in lo, or their weight in both words
  double tab[kExpTab * kExpCopies];    // 2^(j / 32), a copy for each lane of a half-warp: no bank conflicts
  u64 mine[kList];                     // this CTA's part of the list
  u64 list[kList];                     // (ordered key of x, ~id): greater = earlier in the order
  u64 group[kMaxCluster][kGroups];     // every CTA's sums of its groups of bins, written by them
  uint32_t part[kMaxCluster];          // every CTA's share of the list
  u64 xch[2][kMaxCluster][2];  // one pair of words per CTA of the cluster, double-buffered
  u64 res[4];                  // what the CTA that holds a border found (written by it into every CTA)
  u64 wsum[2][kWarps];
  float wmax[kWarps], wmin[kWarps];
  u64 target, before;  // the border sought, and what lies before the bin that it was found in
  uint32_t bin, fill, fill_bin;
  uint64_t bar;
};

// shared memory of one CTA: Smem, then the slice of the row
constexpr size_t kSliceOff = (sizeof(Smem) + 127) & ~size_t(127);

// what the kernels may ask for (the largest slice, 128 KB of float32, fits behind Smem and the walk's tree)
constexpr int kMaxDynSmem = 200 * 1024;

// entries per CTA: a multiple of 8, so that a 16-byte granule belongs to one CTA when rows are aligned
__host__ __device__ inline int slice_len(int vocab, int cluster) { return ((vocab + cluster - 1) / cluster + 7) & ~7; }
__host__ __device__ inline size_t slice_bytes(int vocab, int cluster, int esize) {
  return static_cast<size_t>(slice_len(vocab, cluster)) * esize + 32;
}

// Cluster of `rows` rows or sequences that run side by side: the smallest whose CTAs hold their slice in kSliceGoal
// bytes, so that two of them share an SM and one row's copies run under another's passes; while the SMs are not all
// taken, wider ones shorten the passes (a slice keeps two elements a thread).
constexpr size_t kSliceGoal = 80 * 1024;
inline int cluster_size(long long rows, int vocab, int esize, int sms) {
  int c = 1;
  while (c < kMaxCluster && slice_bytes(vocab, c, esize) > kSliceGoal) c *= 2;
  while (c < kMaxCluster && rows * 2 * c <= sms && slice_len(vocab, c) > 2 * kThreads) c *= 2;
  return c;
}

// Sets the attributes of a kernel of this file's users the first time it is launched on a device; the SM count, or -1.
template <typename K>
inline int prepare_kernel(K kernel, std::atomic<int> (&sms_of)[kMaxDevices]) {
  const int dev = current_device();
  if (dev < 0) return -1;
  int sms = sms_of[dev].load(std::memory_order_acquire);
  if (sms == 0) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynSmem) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return -1;
    sms_of[dev].store(sms, std::memory_order_release);
  }
  return sms;
}

__device__ __forceinline__ uint32_t ord32(float x) {  // a < b iff ord32(a) < ord32(b); -0 counts as +0
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float ord32_value(uint32_t k) { return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k); }

struct RowParams {
  double t, inv_t;    // T, 1 / T (1 when greedy)
  double ln_min_p_t;  // T ln(min_p), -inf when off
  double top_p;
  int top_k;
  bool greedy;
};

// Reads and checks the parameters of row r; false if one is out of range.
__device__ __forceinline__ bool read_params(const SampleParams& sp, long long r, RowParams& p) {
  const float t = __ldg(sp.temperature + r);
  const int k = sp.top_k != nullptr ? __ldg(sp.top_k + r) : 0;
  const float tp = sp.top_p != nullptr ? __ldg(sp.top_p + r) : 1.f;
  const float mp = sp.min_p != nullptr ? __ldg(sp.min_p + r) : 0.f;
  if (!(t >= 0.f) || isinf(t) || k < 0 || !(tp >= 0.f && tp <= 1.f) || !(mp >= 0.f && mp <= 1.f)) return false;
  p.greedy = t == 0.f;
  p.t = p.greedy ? 1.0 : static_cast<double>(t);
  p.inv_t = 1.0 / p.t;
  p.ln_min_p_t = mp > 0.f ? static_cast<double>(t) * log(static_cast<double>(mp)) : -INFINITY;
  p.top_p = tp;
  p.top_k = k;
  return true;
}
__device__ __forceinline__ bool good_u(float u) { return u >= 0.f && u < 1.f; }

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

// Descending sort of the first n2 (a power of two) entries of a list by all threads of the CTA.
__device__ __forceinline__ void sort_desc(u64* a, int n2) {
  const int tid = threadIdx.x;
  if (n2 <= 64) {  // one warp
    if (tid < 32) {
      for (int k = 2; k <= n2; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
          const int i = ((tid & ~(j - 1)) << 1) | (tid & (j - 1));
          if (i + j < n2) {
            const u64 x = a[i], y = a[i + j];
            if ((x < y) == ((i & k) == 0)) {
              a[i] = y;
              a[i + j] = x;
            }
          }
          __syncwarp();
        }
    }
    __syncthreads();
    return;
  }
  for (int k = 2; k <= n2; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      const int i = ((tid & ~(j - 1)) << 1) | (tid & (j - 1));
      if (i + j < n2) {
        const u64 x = a[i], y = a[i + j];
        if ((x < y) == ((i & k) == 0)) {
          a[i] = y;
          a[i + j] = x;
        }
      }
      __syncthreads();
    }
}

// One CTA's view of the row.  Every member function is called by all threads of all CTAs of the cluster, in the same
// order; the decisions between them follow from values that every CTA holds alike.
template <typename T>
struct Row {
  static constexpr int kPer = Granule<T>::n;
  Smem& s;
  uint8_t* buf;
  int rank, C, tid, lane, warp;
  int vocab, fx;
  int grans;    // 16-byte granules of the slice
  int id0;      // token id of the first element of granule 0 (elements outside the slice hold -inf)
  float m, least;  // largest and smallest candidate
  double md, c32, magic;
  float x_zero;  // below it weights round to 0
  float cut_x;   // the set kept so far
  int cut_id;
  float top;     // this thread's largest element
  bool flat;     // m = +inf: every candidate is +inf and weighs the same
  int parity = 0;

  __device__ Row(Smem& smem, uint8_t* slice, int rank_, int c, int vocab_)
      : s(smem), buf(slice), rank(rank_), C(c), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5),
        vocab(vocab_) {
    const int lg = vocab > 1 ? 32 - __clz(vocab - 1) : 0;
    fx = min(48, 62 - lg);
    magic = __hiloint2double((1023 + 52 - fx) << 20, 0);  // 2^(52 - fx)
    static_assert(kThreads == kExpTab * kExpCopies && kExpTab == 32 && kExpCopies == 16, "one entry per thread");
    s.tab[tid] = g_exp2_frac128[4 * (tid / kExpCopies)];
    if (tid == 0) {
      mbar_init(&s.bar, 1);
      fence_barrier_init();
    }
  }

  __device__ __forceinline__ u64 one() const { return 1ull << fx; }
  // round(2^fx exp((x - m) / T)) for x_zero <= x <= m, from the mantissa of exp + 2^(52 - fx).  With
  // (x - m) / T = (n + r) ln2 / 32, n integer and |r| <= 1/2, exp = 2^(n >> 5) 2^((n & 31) / 32) e^(r ln2 / 32), the
  // last factor by its Taylor series through the fifth power (truncation below 2^-48).  Exactly 2^fx at x = m.
  // A table of 512 entries needs three terms only, but its lookups conflict (6 a clock and SM against 16 here).
  __device__ __forceinline__ u64 weight(float x) const {
    if (flat) return one();
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
    return static_cast<u64>(__double_as_longlong(fma(s2, p, magic)) - __double_as_longlong(magic));
  }
  __device__ __forceinline__ bool kept(float x, int id) const { return x > cut_x || (x == cut_x && id <= cut_id); }
  __device__ __forceinline__ int id_of(int g, int e) const { return id0 + g * kPer + e; }
  __device__ __forceinline__ void read(int g, float (&x)[kPer]) const {
    Granule<T>::unpack(reinterpret_cast<const uint4*>(buf)[g], x);
  }
  // The kept weights of granule g (0 for the others), computed side by side; false if there are none.
  __device__ __forceinline__ bool weights(int g, float (&x)[kPer], u64 (&w)[kPer]) const {
    read(g, x);
    bool take[kPer], any = false;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      take[e] = kept(x[e], id_of(g, e)) && x[e] >= x_zero;
      any = any || take[e];
      w[e] = 0;
    }
    if (!any) return false;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const u64 v = weight(take[e] ? x[e] : m);
      w[e] = take[e] ? v : 0;
    }
    return true;
  }

  // Starts the copy of this CTA's slice of the row; the base of the logits is 16-byte aligned, so the granule that
  // the slice starts in belongs to them.
  __device__ void start(const T* row) {
    const int per = slice_len(vocab, C);
    const int lo = min(vocab, rank * per), hi = min(vocab, lo + per);
    const uintptr_t a = reinterpret_cast<uintptr_t>(row + lo);
    const int head = static_cast<int>(a & 15);
    const int bytes = lo < hi ? head + (hi - lo) * static_cast<int>(sizeof(T)) : 0;
    const int full = bytes >> 4;
    grans = (bytes + 15) >> 4;
    id0 = lo - head / static_cast<int>(sizeof(T));
    if (tid == 0) {
      mbar_arrive_expect_tx(&s.bar, full * 16);
      if (full > 0)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                smem_u32(buf)),
            "l"(a - head), "r"(full * 16), "r"(smem_u32(&s.bar))
            : "memory");
    }
    // the last granule's elements, when the slice ends inside one
    T* tail = reinterpret_cast<T*>(buf) + full * kPer;
    if (full < grans && tid < kPer) {
      const int id = id0 + full * kPer + tid;
      tail[tid] = id < hi ? row[id] : static_cast<T>(-INFINITY);
    }
  }
  // Brings this CTA's slice of a row into L2 (whole granules inside the row).
  __device__ void prefetch(const T* row) const {
    const int per = slice_len(vocab, C);
    const int lo = min(vocab, rank * per), hi = min(vocab, lo + per);
    const uintptr_t a = (reinterpret_cast<uintptr_t>(row + lo) + 15) & ~uintptr_t(15);
    const uintptr_t e = reinterpret_cast<uintptr_t>(row + hi) & ~uintptr_t(15);
    if (a < e)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"(static_cast<uint32_t>(e - a)) : "memory");
  }
  // Waits for it (bounded) and clears what lies before the slice in its first granule.
  __device__ bool finish(uint32_t phase) {
    volatile int never = 0;
    const bool ok = mbar_wait(&s.bar, phase, &never);
    const int per = slice_len(vocab, C), lo = min(vocab, rank * per);
    if (grans > 0 && tid < lo - id0) reinterpret_cast<T*>(buf)[tid] = static_cast<T>(-INFINITY);
    return __syncthreads_and(ok);
  }

  // Every CTA's pair of words, in s.xch[result] afterwards; a and b need to be valid in threads 0 .. C-1.
  __device__ int exchange(u64 a, u64 b) {
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
  __device__ bool find_range(bool ok) {
    float mx = -INFINITY, mn = INFINITY;
    for (int g = tid; g < grans; g += kThreads) {
      float x[kPer];
      read(g, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        mx = fmaxf(mx, x[e]);  // NaN drops out
        mn = fminf(mn, x[e] == -INFINITY ? INFINITY : x[e]);
      }
    }
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
    flat = m == INFINITY;
    return all;
  }

  // Exclusive prefix of (a, b) over the CTA's threads and the CTA's totals.
  __device__ void block_scan(u64 a, u64 b, u64& ea, u64& eb, u64& ta, u64& tb) {
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
  __device__ void clear_bins() {
    for (int i = tid; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0;
    __syncthreads();
  }

  // Bins in the order of the candidates: bin 0 holds the largest.
  float bin_scale;
  __device__ __forceinline__ int bin_of(float x) const {
    const float d = fminf((m - x) * bin_scale, static_cast<float>(kBins - 1));
    return __float_as_int(d + 12582912.f) & 0x7fffff & (2 * kBins - 1);  // rint(d), by adding 1.5 * 2^23
  }
  __device__ void set_bins(const RowParams& rp) {
    const float span = fminf(static_cast<float>(kBinRange * rp.t), m - least);
    bin_scale = span > 0.f ? fminf(static_cast<float>(kBins - 1) / span, 1e37f) : 0.f;
  }

  // Fills the histogram with the kept elements and finds the bin that holds element number k (mass false) or at which
  // the running weight reaches the share top_p of the whole (mass true): s.bin, s.target and what lies before the bin.
  // false, with no bin, if there are no more than k elements.
  __device__ bool find_bin(bool mass, u64 k, double share) {
    clear_bins();
    for (int g = tid; g < grans; g += kThreads) {
      float x[kPer];
      if (mass) {
        u64 w[kPer];
        if (!weights(g, x, w)) continue;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (w[e] != 0) add_mass(bin_of(x[e]), w[e]);
      } else {
        read(g, x);
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (kept(x[e], id_of(g, e))) atomicAdd(&s.lo[bin_of(x[e])], 1u);
      }
    }
    __syncthreads();
    cg::cluster_group cl = cg::this_cluster();
    // the sums of this CTA's groups of bins go to every CTA
    for (int g = warp; g < kGroups; g += kWarps) {
      u64 w = s.lo[g * 32 + lane] | static_cast<u64>(s.hi[g * 32 + lane]) << 32;
      w = warp_sum_u64(w);
      if (lane < C) *cl.map_shared_rank(&s.group[rank][g], lane) = w;
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
        u64 v[kMaxCluster], fw = 0;  // lane = bin of that group; all CTAs' loads in flight at once
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          v[c] = 0;
          if (c < C)
            v[c] = *cl.map_shared_rank(&s.lo[grp * 32 + lane], c) |
                   static_cast<u64>(*cl.map_shared_rank(&s.hi[grp * 32 + lane], c)) << 32;
        }
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) fw += v[c];
        const u64 fiw = w0 + warp_incl_u64(fw, lane);
        const int at = __ffs(__ballot_sync(0xffffffffu, fiw >= target)) - 1;
        if (lane == at) {
          s.bin = grp * 32 + at;
          s.before = fiw - fw;
        }
      } else if (lane == 0) {
        s.bin = kBins;
      }
      if (lane == 0) s.target = target;
    }
    __syncthreads();
    return s.bin < kBins;
  }

  // Writes this CTA's kept elements of bin `last`, and with `whole` of the bins before it, to s.mine (as many as fit);
  // s.fill counts them, s.fill_bin those of `last`.
  __device__ void gather(int last, bool whole) {
    __syncthreads();
    if (tid == 0) s.fill = s.fill_bin = 0;
    __syncthreads();
    for (int g = tid; g < grans; g += kThreads) {
      float x[kPer];
      read(g, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (!kept(x[e], id_of(g, e))) continue;
        const int b = bin_of(x[e]);
        if (b > last || (!whole && b != last)) continue;
        if (b == last) atomicAdd(&s.fill_bin, 1u);
        const uint32_t at = atomicAdd(&s.fill, 1u);
        if (at < kList) s.mine[at] = static_cast<u64>(ord32(x[e])) << 32 | static_cast<uint32_t>(~id_of(g, e));
      }
    }
    __syncthreads();
  }
  // Joins the n entries that the CTAs hold together (this one's from `base` on) in every CTA, in order.
  __device__ void join(int base, int n) {
    for (int i = tid; i < static_cast<int>(s.fill) * C; i += kThreads)
      *cg::this_cluster().map_shared_rank(&s.list[base + i / C], i % C) = s.mine[i / C];
    cg::this_cluster().sync();
    order(n);
  }
  __device__ void order(int n) {
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
    int n2 = 2;
    while (n2 < n) n2 *= 2;
    if (tid < n2 - n) s.list[n + tid] = 0;  // n2 - n < kThreads
    __syncthreads();
    sort_desc(s.list, n2);
  }

  // Lists what is kept up to the bin found, or that bin alone (whole becomes false), in every CTA and in order; the
  // number, 0 if even that is more than a list holds.
  __device__ int list_bin(bool& whole) {
    const int last = static_cast<int>(s.bin);
    gather(last, true);
    for (;;) {
      const int p = exchange(s.fill, s.fill_bin);
      u64 n = 0, base = 0, n_bin = 0;
      for (int c = 0; c < C; ++c) {
        if (c < rank) base += s.xch[p][c][0];
        n += s.xch[p][c][0];
        n_bin += s.xch[p][c][1];
      }
      if (n <= kList) {
        join(static_cast<int>(base), static_cast<int>(n));
        return static_cast<int>(n);
      }
      if (!whole || n_bin > kList) return 0;
      whole = false;
      gather(last, false);
    }
  }

  // Lists a superset of the k largest kept elements in every CTA, in order, from each CTA's elements that are no
  // smaller than the k-th largest of its thread maxima; the number, or 0 if that does not work out (k too large, ties).
  __device__ int list_largest(int k) {
    const int room = kList / C;
    if (k > room || k > kThreads / 2) return 0;
    clear_bins();
    if (tid == 0) s.bin = kBins - 1;  // fewer than k threads have a candidate: all elements
    if (kept(top, -1)) atomicAdd(&s.lo[bin_of(top)], 1u);
    __syncthreads();
    if (warp == 0) {
      uint32_t n = 0;  // lane = group of bins
      for (int i = 0; i < 32; ++i) n += s.lo[lane * 32 + ((i + lane) & 31)];
      uint32_t in = static_cast<uint32_t>(warp_incl_u64(n, lane));
      const uint32_t hit = __ballot_sync(0xffffffffu, in >= static_cast<uint32_t>(k));
      if (hit != 0) {
        const int grp = __ffs(hit) - 1;
        const uint32_t n0 = __shfl_sync(0xffffffffu, in - n, grp);
        in = n0 + static_cast<uint32_t>(warp_incl_u64(s.lo[grp * 32 + lane], lane));
        const int at = __ffs(__ballot_sync(0xffffffffu, in >= static_cast<uint32_t>(k))) - 1;
        if (lane == 0) s.bin = grp * 32 + at;
      }
    }
    __syncthreads();
    gather(static_cast<int>(s.bin), true);
    const bool fits = s.fill <= static_cast<uint32_t>(room);
    if (tid < C) *cg::this_cluster().map_shared_rank(&s.part[rank], tid) = s.fill;
    if (fits)
      for (int i = tid; i < static_cast<int>(s.fill) * C; i += kThreads)
        *cg::this_cluster().map_shared_rank(&s.list[rank * room + i / C], i % C) = s.mine[i / C];
    cg::this_cluster().sync();
    // the parts move together; what lies behind the last is cleared
    int n = 0, most = 0;
    for (int c = 0; c < C; ++c) {
      n += s.part[c];
      most = max(most, static_cast<int>(s.part[c]));
    }
    if (most > room) return 0;
    u64 v[kList / kThreads];
    int to[kList / kThreads];
#pragma unroll
    for (int i = 0; i < kList / kThreads; ++i) {
      const int from = tid + i * kThreads, c = from / room, at = from % room;
      to[i] = -1;
      if (at < static_cast<int>(s.part[c])) {
        v[i] = s.list[from];
        to[i] = at;
        for (int b = 0; b < c; ++b) to[i] += s.part[b];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kList / kThreads; ++i)
      if (to[i] >= 0) s.list[to[i]] = v[i];
    __syncthreads();
    order(n);
    return n;
  }
  __device__ __forceinline__ float list_x(int i) const { return ord32_value(static_cast<uint32_t>(s.list[i] >> 32)); }
  __device__ __forceinline__ int list_id(int i) const { return static_cast<int>(~static_cast<uint32_t>(s.list[i])); }
  __device__ __forceinline__ u64 list_weight(int i) const {
    const float x = list_x(i);
    return x >= x_zero ? weight(x) : 0;
  }

  // Index of the first of the list's n elements at which the running weight reaches `target`, which it does.
  __device__ int list_border(int n, u64 target) {
    const u64 a = 2 * tid < n ? list_weight(2 * tid) : 0, b = 2 * tid + 1 < n ? list_weight(2 * tid + 1) : 0;
    u64 before, e2, total, t2;
    block_scan(a + b, 0, before, e2, total, t2);
    if (before < target && target <= before + a) s.fill = 2 * tid;
    else if (before + a < target && target <= before + a + b) s.fill = 2 * tid + 1;
    __syncthreads();
    return static_cast<int>(s.fill);
  }
  __device__ u64 list_mass(int n) {
    const u64 a = 2 * tid < n ? list_weight(2 * tid) : 0, b = 2 * tid + 1 < n ? list_weight(2 * tid + 1) : 0;
    u64 e1, e2, total, t2;
    block_scan(a + b, 0, e1, e2, total, t2);
    return total;
  }

  // The draw among the first n elements of the list: the first, by id, whose running weight exceeds u times all.
  __device__ void draw_from_list(int n, float u, Drawn& d) {
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
      int n2 = 2;
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
    const double y = flat ? 0.0 : (static_cast<double>(x) - md) * (c32 * (0.69314718055994530942 / kExpTab));
    return static_cast<float>(y - (log(static_cast<double>(total)) - fx * 0.69314718055994530942));
  }

  // Narrows the kept set to end at its element number `k` (mass false), or at the element where the running weight
  // reaches `target` (mass true), whatever the values: an interval of keys is narrowed by histograms to one key.  The set
  // is known to hold that much.
  __device__ void cut_by_key(bool mass, u64 target) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();  // no CTA reads the last histogram any more
    uint32_t base = ord32(m);
    int bits = 32;  // the interval is (base - 2^bits, base]
    while (bits > 0) {
      const int shift = bits > kBinBits ? bits - kBinBits : 0;
      clear_bins();
      for (int g = tid; g < grans; g += kThreads) {
        float x[kPer];
        read(g, x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (!kept(x[e], id_of(g, e))) continue;
          const uint32_t d = base - ord32(x[e]);  // wraps for keys above the interval
          if (bits < 32 && (d >> bits) != 0) continue;
          if (!mass) atomicAdd(&s.lo[d >> shift], 1u);
          else if (x[e] >= x_zero) add_mass(d >> shift, weight(x[e]));
        }
      }
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
    find_id<true>(nth - 1, -1.0, [&](int g, float(&x)[kPer], u64(&w)[kPer]) {
      read(g, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) w[e] = x[e] == v && kept(x[e], id_of(g, e)) ? 1 : 0;
    }, total, id, at);
    cut_x = v;
    cut_id = id;
  }

  // The lowest id at which the running sum of f, in id order, exceeds t, and its value; t is `fixed` if share < 0, else
  // floor(share * total).  f(g, x, w) gives the values and terms of granule g.  kAll: every thread of the cluster gets
  // the result; otherwise the thread that returns true does, and all get the total.
  template <bool kAll, typename F>
  __device__ bool find_id(u64 fixed, double share, F f, u64& total, int& id, float& at) {
    // warp w owns granules [w * gw, (w + 1) * gw): ids ascend over warps, iterations and lanes
    const int gw = (((grans + kWarps - 1) / kWarps) + 31) & ~31;
    const int g0 = min(grans, warp * gw), g1 = min(grans, g0 + gw);
    u64 sum = 0;
    for (int g = g0 + lane; g < g1; g += 32) {
      float x[kPer];
      u64 w[kPer];
      f(g, x, w);
#pragma unroll
      for (int e = 0; e < kPer; ++e) sum += w[e];
    }
    sum = warp_sum_u64(sum);
    __syncthreads();
    if (lane == 0) s.wsum[0][warp] = sum;
    __syncthreads();
    u64 mine = 0, before = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s.wsum[0][w];
      mine += s.wsum[0][w];
    }
    const int p = exchange(mine, 0);
    total = 0;
    for (int c = 0; c < C; ++c) {
      if (c < rank) before += s.xch[p][c][0];
      total += s.xch[p][c][0];
    }
    const u64 t = share < 0 ? fixed : static_cast<u64>(share * static_cast<double>(total));
    bool found = false;
    if (before <= t && t < before + sum) {  // one warp of the cluster
      u64 run = before;
      for (int gb = g0; gb < g1; gb += 32) {
        const int g = gb + lane;
        float x[kPer];
        u64 w[kPer], mysum = 0;
        if (g < g1) f(g, x, w);
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

  // The draw among the first n elements of the list, or with by_p their shortest prefix of the share top_p.
  __device__ void draw_from_largest(bool by_p, double top_p, int n, float u, Drawn& d) {
    if (by_p) {
      const u64 all = list_mass(n), want = static_cast<u64>(ceil(top_p * static_cast<double>(all)));
      n = 1 + list_border(n, want < 1 ? 1 : (want > all ? all : want));
    }
    draw_from_list(n, u, d);
  }
  // The kept set ends at entry `at` of the list.
  __device__ void cut_at(int at) {
    cut_x = list_x(at);
    cut_id = list_id(at);
    __syncthreads();
  }

  // The whole draw from the slice that start() is bringing in.  kAll: the result is wanted in every thread; otherwise in
  // the one whose result says so (and CTAs may return from here while others still work on their own).
  template <bool kAll>
  __device__ Drawn draw(const RowParams& rp, float u, uint32_t phase) {
    Drawn d{-1, -INFINITY, true, rank == 0 && tid == 0};
    d.ok = find_range(finish(phase));
    if (!d.ok || m == -INFINITY) return d;
    c32 = rp.inv_t * (kExpTab / 0.69314718055994530942);
    x_zero = __double2float_rd(md - (fx + 2) * 0.69314718055994530942 * rp.t);
    cut_id = INT_MAX;
    cut_x = rp.greedy || flat ? m : fmaxf(__double2float_ru(md + rp.ln_min_p_t), -3.402823466e38f);
    set_bins(rp);
    if (!rp.greedy) {
      // top-k by the count, then top-p by the weight; a list that holds all that is kept ends the draw
      const bool by_k = rp.top_k > 0 && rp.top_k < vocab, by_p = rp.top_p < 1.0;
      bool whole = true;
      int n = by_k && !flat ? list_largest(rp.top_k) : 0;
      if (n > 0) {
        if (!kAll && rank != 0) return d;
        n = min(n, rp.top_k);
        draw_from_largest(by_p, rp.top_p, n, u, d);
        return d;
      }
      if (by_k && find_bin(false, rp.top_k, 0.0)) {
        const u64 before = s.before;
        n = list_bin(whole);
        if (n > 0 && whole) {
          if (!kAll && rank != 0) return d;
          draw_from_largest(by_p, rp.top_p, rp.top_k, u, d);
          return d;
        }
        if (n > 0) cut_at(static_cast<int>(rp.top_k - before) - 1);
        else cut_by_key(false, rp.top_k);
      }
      if (by_p) {
        whole = true;
        if (by_k) cg::this_cluster().sync();  // no CTA reads the last histogram or its list's parts any more
        find_bin(true, 0, rp.top_p);
        const u64 before = s.before, target = s.target;
        n = list_bin(whole);
        if (n > 0 && whole) {
          if (!kAll && rank != 0) return d;
          n = 1 + list_border(n, target);
          draw_from_list(n, u, d);
          return d;
        }
        if (n > 0) cut_at(list_border(n, target - before));
        else cut_by_key(true, target);
      }
    }
    u64 total;
    const bool found = find_id<kAll>(0, rp.greedy ? 0.0 : static_cast<double>(u),
                                     [&](int g, float(&x)[kPer], u64(&w)[kPer]) { weights(g, x, w); }, total, d.token,
                                     d.logprob);
    if (!kAll) d.mine = found;
    d.logprob = rp.greedy ? 0.f : log_prob(d.logprob, total);
    return d;
  }
};

}  // namespace smp
}  // namespace jf
