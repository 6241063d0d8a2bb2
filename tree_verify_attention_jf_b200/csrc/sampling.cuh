// sampling.cuh -- drawing a token from one row of logits that lies in the shared memory of a thread-block cluster.
//
// Mathematics.  With w_v = exp((x_v - m) / T) the filters min-p, top-k and top-p each keep a prefix of the candidates in
// the order (x descending, id ascending), so the set kept is described by one cut (cut_x, cut_id): v is kept iff
// x_v > cut_x, or x_v == cut_x and v <= cut_id.  min-p is a cut at a value.  The top-k cut is the element of a given
// rank, the top-p cut the element at which the running weight reaches a given mass; both are found without sorting, by
// histograms over the order-preserving integer image of x that narrow an interval of keys down to one value, then
// by id among the equal ones.  The draw itself is an inverse CDF over the kept weights in id order.
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

// 2^(j/128) for the float64 exp (each translation unit keeps its own copy)
static __device__ const double g_exp2_frac128[128] = JF_EXP2_FRAC128;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBinBits = 11;
constexpr int kBins = 1 << kBinBits;

struct Smem {
  uint32_t cnt[kBins], lo[kBins], hi[kBins];  // histogram: elements, and their weight in two words
  double tab[128];
  u64 xch[2][kMaxCluster][2];  // one pair of words per CTA of the cluster, double-buffered
  u64 res[5];                  // what the CTA that holds a border found (written by it into every CTA)
  u64 wsum[2][kWarps];
  u64 pair[2];
  float wmax[kWarps];
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

__device__ __forceinline__ uint32_t ord32(float x) {  // a < b iff ord32(a) < ord32(b); -0 counts as +0
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float ord32_value(uint32_t k) { return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k); }

struct RowParams {
  double inv_t;  // 1 / T
  double ln_min_p_t;  // T ln(min_p), -inf when off
  double top_p;
  float u;
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
  p.inv_t = p.greedy ? 1.0 : 1.0 / static_cast<double>(t);
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
};

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
  float m;
  double md, inv_t;
  float cut_x;  // the set kept so far
  int cut_id;
  int parity = 0;

  __device__ Row(Smem& smem, uint8_t* slice, int rank_, int c, int vocab_)
      : s(smem), buf(slice), rank(rank_), C(c), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5),
        vocab(vocab_) {
    const int lg = vocab > 1 ? 32 - __clz(vocab - 1) : 0;
    fx = min(48, 62 - lg);
  }

  __device__ __forceinline__ u64 one() const { return 1ull << fx; }
  // round(2^fx exp((x - m) / T)) from the mantissa of exp + 2^(52 - fx)
  __device__ __forceinline__ u64 weight(float x) const {
    if (x == m) return one();
    const double w = exp_nonpos_f64((static_cast<double>(x) - md) * inv_t, s.tab);
    const double magic = __hiloint2double((1023 + 52 - fx) << 20, 0);
    return static_cast<u64>(__double_as_longlong(w + magic) - __double_as_longlong(magic));
  }
  __device__ __forceinline__ bool kept(float x, int id) const { return x > cut_x || (x == cut_x && id <= cut_id); }
  __device__ __forceinline__ int id_of(int g, int e) const { return id0 + g * kPer + e; }
  __device__ __forceinline__ void read(int g, float (&x)[kPer]) const {
    Granule<T>::unpack(reinterpret_cast<const uint4*>(buf)[g], x);
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

  // The row's maximum; s.tab is filled on the way.  -inf if there is no candidate.
  __device__ bool find_max(bool ok) {
    float mx = -INFINITY;
    for (int g = tid; g < grans; g += kThreads) {
      float x[kPer];
      read(g, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) mx = fmaxf(mx, x[e]);  // NaN drops out
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) s.wmax[warp] = mx;
    __syncthreads();
    mx = s.wmax[lane & (kWarps - 1)];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const int p = exchange(__float_as_uint(mx), ok ? 1 : 0);
    bool all = true;
    m = -INFINITY;
    for (int c = 0; c < C; ++c) {
      m = fmaxf(m, __uint_as_float(static_cast<uint32_t>(s.xch[p][c][0])));
      all = all && s.xch[p][c][1] != 0;
    }
    md = static_cast<double>(m);
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

  // Narrows the kept set to end at its element number `k` (mass false), or at the element where the running weight
  // reaches `share` of the whole kept weight (mass true).
  __device__ void cut(bool mass, u64 k, double share) {
    uint32_t khi = ord32(m);
    u64 target = k;    // of what is still to be found inside the interval of keys
    uint32_t base = khi;
    int bits = 32;     // the interval is (base - 2^bits, base]
    for (int level = 0; bits > 0; ++level) {
      const int shift = bits > kBinBits ? bits - kBinBits : 0;
      for (int i = tid; i < kBins; i += kThreads) s.cnt[i] = s.lo[i] = s.hi[i] = 0;
      __syncthreads();
      for (int g = tid; g < grans; g += kThreads) {
        float x[kPer];
        read(g, x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (!kept(x[e], id_of(g, e))) continue;
          const uint32_t d = base - ord32(x[e]);  // wraps for keys above the interval
          if (bits < 32 && (d >> bits) != 0) continue;
          const int bin = d >> shift;
          if (mass) {
            const u64 w = weight(x[e]);
            const uint32_t add = static_cast<uint32_t>(w), old = atomicAdd(&s.lo[bin], add);
            const uint32_t up = static_cast<uint32_t>(w >> 32) + (old + add < old ? 1u : 0u);
            if (up != 0) atomicAdd(&s.hi[bin], up);
          } else {
            atomicAdd(&s.cnt[bin], 1u);
          }
        }
      }
      cg::cluster_group cl = cg::this_cluster();
      cl.sync();  // every CTA's histogram is complete
      // this CTA sums its share of the bins over the cluster: consecutive bins per thread, in order
      const int seg = (kBins + C - 1) / C, b0 = rank * seg, b1 = min(kBins, b0 + seg);
      const int per = (seg + kThreads - 1) / kThreads;
      const int t0 = b0 + tid * per;
      u64 sum = 0;
      u64 v[kBins / kThreads];
#pragma unroll
      for (int i = 0; i < kBins / kThreads; ++i) {
        v[i] = 0;
        if (i < per && t0 + i < b1) {
          for (int c = 0; c < C; ++c) {
            if (mass) {
              v[i] += *cl.map_shared_rank(&s.lo[t0 + i], c);
              v[i] += static_cast<u64>(*cl.map_shared_rank(&s.hi[t0 + i], c)) << 32;
            } else {
              v[i] += *cl.map_shared_rank(&s.cnt[t0 + i], c);
            }
          }
          sum += v[i];
        }
      }
      u64 excl, e2, total, t2;
      block_scan(sum, 0, excl, e2, total, t2);
      const int p = exchange(total, 0);
      u64 before = 0, all = 0;
      for (int c = 0; c < C; ++c) {
        if (c < rank) before += s.xch[p][c][0];
        all += s.xch[p][c][0];
      }
      if (level == 0) {
        if (mass) {
          target = static_cast<u64>(ceil(share * static_cast<double>(all)));
          target = target < 1 ? 1 : (target > all ? all : target);
        } else if (all <= k) {
          return;  // no more candidates than that
        }
      }
      u64 run = before + excl;
#pragma unroll
      for (int i = 0; i < kBins / kThreads; ++i) {
        if (run < target && target <= run + v[i]) {  // exactly one thread of the cluster
          for (int c = 0; c < C; ++c) {
            u64* r = cl.map_shared_rank(&s.res[0], c);
            r[0] = t0 + i;
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
    const int id = find_id(nth - 1, 0.0, [&](float x, int i) { return x == v && kept(x, i) ? u64(1) : u64(0); }, nullptr);
    cut_x = v;
    cut_id = id;
  }

  // The lowest id at which the running sum of f(x, id), in id order, exceeds t; t is `fixed`, or with total given
  // floor(share * sum) and *total becomes the sum.  -1 if there is none.
  template <typename F>
  __device__ int find_id(u64 fixed, double share, F f, u64* total) {
    // warp w owns granules [w * gw, (w + 1) * gw): ids ascend over warps, iterations and lanes
    const int gw = (((grans + kWarps - 1) / kWarps) + 31) & ~31;
    const int g0 = min(grans, warp * gw), g1 = min(grans, g0 + gw);
    u64 sum = 0;
    for (int g = g0 + lane; g < g1; g += 32) {
      float x[kPer];
      read(g, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) sum += f(x[e], id_of(g, e));
    }
    sum = warp_sum_u64(sum);
    __syncthreads();
    if (lane == 0) s.wsum[0][warp] = sum;
    if (tid == 0) s.res[2] = ~0ull;
    __syncthreads();
    u64 mine = 0, before_warp = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before_warp += s.wsum[0][w];
      mine += s.wsum[0][w];
    }
    const int p = exchange(mine, 0);
    u64 before = before_warp, all = 0;
    for (int c = 0; c < C; ++c) {
      if (c < rank) before += s.xch[p][c][0];
      all += s.xch[p][c][0];
    }
    const u64 t = total != nullptr ? static_cast<u64>(share * static_cast<double>(all)) : fixed;
    if (total != nullptr) *total = all;
    if (before <= t && t < before + sum) {  // one warp of the cluster
      u64 run = before;
      for (int gb = g0; gb < g1; gb += 32) {
        const int g = gb + lane;
        float x[kPer];
        u64 w[kPer], mysum = 0;
        if (g < g1) read(g, x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          w[e] = g < g1 ? f(x[e], id_of(g, e)) : 0;
          mysum += w[e];
        }
        const u64 incl = run + warp_incl_u64(mysum, lane);
        const uint32_t hit = __ballot_sync(0xffffffffu, incl > t);
        if (hit != 0) {
          if (lane == __ffs(hit) - 1) {
            u64 r = incl - mysum;
            int at = 0;
#pragma unroll
            for (int e = kPer - 1; e >= 0; --e) {
              u64 through = r;
              for (int i = 0; i <= e; ++i) through += w[i];
              if (through > t) at = e;
            }
            for (int c = 0; c < C; ++c) {
              u64* dst = cg::this_cluster().map_shared_rank(&s.res[2], c);
              dst[0] = static_cast<u64>(id_of(g, at));
              dst[1] = __float_as_uint(x[at]);
            }
          }
          break;
        }
        run = __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    cg::this_cluster().sync();
    return static_cast<int>(static_cast<long long>(s.res[2]));
  }

  // The whole draw from the slice that start() is bringing in.
  __device__ Drawn draw(const RowParams& rp, float u, uint32_t phase) {
    Drawn d{-1, -INFINITY, true};
    inv_t = rp.inv_t;
    d.ok = find_max(finish(phase));
    if (!d.ok || m == -INFINITY) {
      cg::this_cluster().sync();  // nobody leaves while another CTA may still write into its shared memory
      return d;
    }
    cut_id = INT_MAX;
    if (rp.greedy || m == INFINITY) {
      cut_x = m;
    } else {
      const double least = md + rp.ln_min_p_t;
      cut_x = fmaxf(__double2float_ru(least), -3.402823466e38f);
    }
    if (!rp.greedy) {
      if (rp.top_k > 0 && rp.top_k < vocab) cut(false, rp.top_k, 0.0);
      if (rp.top_p < 1.0) cut(true, 0, rp.top_p);
    }
    u64 total = 0;
    d.token = find_id(0, rp.greedy ? 0.0 : static_cast<double>(u),
                      [&](float x, int id) { return kept(x, id) ? weight(x) : u64(0); }, &total);
    const float x = __uint_as_float(static_cast<uint32_t>(s.res[3]));
    const double y = x == m ? 0.0 : (static_cast<double>(x) - md) * inv_t;
    d.logprob = rp.greedy ? 0.f : static_cast<float>(y - (log(static_cast<double>(total)) - fx * 0.69314718055994530942));
    return d;
  }
};

}  // namespace smp
}  // namespace jf
