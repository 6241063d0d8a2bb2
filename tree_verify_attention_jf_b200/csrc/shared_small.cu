// shared_small.cu -- the own keys of sequences with few query rows, for tree attention over a shared prefix (sm_100a).
//
// What it computes: the softmax state (unnormalised O, running max, row sum) of a sequence's rows against the slots
// that it does not share, for sequences whose N tree nodes x g query heads make at most 16 rows and whose own slots are
// few (small_sequence()).  The persistent kernel of tree_attention.cu gives every (sequence, kv head) a pair of 128-row
// M tiles and a pipeline to fill, which for one decoded token and a hundred keys costs far more than the keys' bytes:
// 64 single tokens with 16384 shared and up to 256 own slots (8 kv heads) took 102 us a call without this kernel and
// 75 with it.
//
// Design: bound by latency, then by the cache's bytes.  One CTA of four warps per (sequence, kv head); a warp takes a
// page (16 keys) at a time and multiplies it with mma.sync, whose 16 rows fit the few query rows where a tcgen05 tile
// would be almost empty.  Both products are invariant to a permutation of the contracted index, and the outputs to one
// of the columns, so operands are permuted to let every thread load consecutive bytes straight from the cache: thread t
// of a quad holds elements 32 t .. 32 t + 31 of its key's row, and 16 consecutive dims of its four V rows.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "jf_device.cuh"
#include "serving_internal.h"

namespace jf {
namespace small {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = kSmallRows;

// D += A B, 16 x 8 x 16, both operands f16 (8-bit cache) or bf16
template <bool kF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t f16_of_bf16(uint32_t w) {  // a pair
  const __half2 h = __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t f16_of_e4m3(uint32_t two) {  // exact
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}

// `n` consecutive elements (a multiple of 16) of a cache row as pairs for the MMA
template <bool kFp8, int n>
__device__ __forceinline__ void load_row(const void* cache, long long element, uint32_t (&w)[n / 2]) {
  if (kFp8) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(cache) + element);
#pragma unroll
    for (int i = 0; i < n / 16; ++i) {
      const uint4 v = __ldg(p + i);
      const uint32_t b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[8 * i + 2 * j] = f16_of_e4m3(b[j]);
        w[8 * i + 2 * j + 1] = f16_of_e4m3(b[j] >> 16);
      }
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(cache) + element);
#pragma unroll
    for (int i = 0; i < n / 8; ++i) {
      const uint4 v = __ldg(p + i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads)
    small_kernel(const __nv_bfloat16* __restrict__ q, const void* __restrict__ k_cache,
                 const void* __restrict__ v_cache, const SharedAttnParams p) {
  __shared__ float s_o[kWarps][kRows][kHeadDim + 4];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ int s_parent[kRows];
  __shared__ int s_page[(kSmallKeys + kPageSize - 1) / kPageSize];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kvh = blockIdx.x, b = blockIdx.y;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before this one (which may produce any input)
  // the sequence; malformed offsets or lengths are left to the other kernel, which reports them.  (The loads that do
  // not depend on the group go first.)
  const int off = __ldg(p.tree_offsets + b), N = __ldg(p.tree_offsets + b + 1) - off, P = __ldg(p.prefix_lens + b);
  int lo = 0, hi = p.num_groups - 1;  // the last group that starts at or before b
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.group_offsets + mid) <= b) lo = mid; else hi = mid - 1;
  }
  const int len = __ldg(p.shared_lens + lo);
  if (off < 0 || N <= 0 || off > p.total_nodes - N || len < 0 || P < len) return;
  const int page0 = len / kPageSize, own = P - page0 * kPageSize;
  if (static_cast<long long>(P) + N > static_cast<long long>(p.max_pages) * kPageSize) return;
  if (!small_sequence(N, p.group, own + N)) return;
  const int rows = N * p.group, keys = own + N, pages = (keys + kPageSize - 1) / kPageSize;
  const int32_t* bt = p.block_table + static_cast<long long>(b) * p.max_pages + page0;
  const int t = lane & 3, r0 = lane >> 2, r1 = r0 + 8;  // the quad's thread, and the rows of its fragments
  // Q: k-step kk contracts elements 32 t' + 4 kk .. + 3 of every quad thread t'
  uint32_t qa[8][4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = half ? r1 : r0;
    const long long row = static_cast<long long>(off + r / p.group) * p.hq + kvh * p.group + r % p.group;
    const uint4* src = reinterpret_cast<const uint4*>(q + row * kHeadDim + 32 * t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = r < rows ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
      qa[2 * i][half] = kFp8 ? f16_of_bf16(v.x) : v.x;
      qa[2 * i][2 + half] = kFp8 ? f16_of_bf16(v.y) : v.y;
      qa[2 * i + 1][half] = kFp8 ? f16_of_bf16(v.z) : v.z;
      qa[2 * i + 1][2 + half] = kFp8 ? f16_of_bf16(v.w) : v.w;
    }
  }
  // parents and page ids
  bool bad = false;
  if (tid < N) {
    const int pi = __ldg(p.parent + off + tid);
    bad = pi < -1 || pi >= tid;
    s_parent[tid] = bad ? -1 : pi;
  }
  for (int i = tid; i < pages; i += kThreads) {
    const int id = __ldg(bt + i);
    bad = bad || id < 0 || id >= p.num_pages;
    s_page[i] = id;
  }
  bad = __syncthreads_or(bad);
  const long long li0 = static_cast<long long>(off) * p.group;  // the rows' place among those of the kv head
  if (bad) {
    if (tid == 0 && kvh == 0) report(p.status, JF_ERR_DEVICE_CHECK);
    if (tid < rows) __stcg(p.row_at(0, kvh) + li0 + tid, make_int4(kRowBad, 0, 0, 0));
    return;
  }
  // which of the (at most 16) tree nodes the two rows see: their root paths
  uint32_t sees[2] = {0, 0};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    int j = (half ? r1 : r0) < rows ? (half ? r1 : r0) / p.group : -1;
    for (int step = 0; step < kRows && j >= 0; ++step) {
      sees[half] |= 1u << j;
      j = s_parent[j];
    }
  }
  float o[16][4];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  for (int pg = warp; pg < pages; pg += kWarps) {
    const long long slot0 = static_cast<long long>(s_page[pg]) * kPageSize;
    const int left = keys - pg * kPageSize;  // keys of this page that exist
    auto element = [&](int key) { return ((slot0 + key) * p.hkv + kvh) * kHeadDim; };
    // K of keys 0-7 and 8-15: column (lane / 4) of each half is this thread's key.  V of keys 2 t, 2 t + 1, 2 t + 8 and
    // 2 t + 9, dims 16 (lane / 4) .. + 15; all loads of the page are in flight together.
    uint32_t kw[2][16], vw[4][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) load_row<kFp8, 32>(k_cache, element(8 * h + r0) + 32 * t, kw[h]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_row<kFp8, 16>(v_cache, element(2 * t + (i & 1) + 8 * (i >> 1)) + 16 * r0, vw[i]);
    float s[2][4];  // S = Q K^T
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) mma<kFp8>(s[h], qa[kk], kw[h][2 * kk], kw[h][2 * kk + 1]);
    }
    // V rows that do not exist count as 0, so that what lies there cannot reach the output through 0 * V
    if (left < kPageSize) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (2 * t + (i & 1) + 8 * (i >> 1) >= left) vw[i][j] = 0;
    }
    // mask, running max and sum per row (values 0, 1: row r0; 2, 3: row r1; keys 2 t, 2 t + 1 of each half)
    uint32_t pa[4];
    float scale[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float y[4];
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = pg * kPageSize + 2 * t + (i & 1) + 8 * (i >> 1), node = key - own;
        const bool vis = node < 0 || (node < N && ((sees[half] >> node) & 1u));
        y[i] = vis ? s[i >> 1][2 * half + (i & 1)] * p.scale_log2 : -INFINITY;
        top = fmaxf(top, y[i]);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float mn = fmaxf(m[half], top), ref = mn == -INFINITY ? 0.f : mn;
      scale[half] = ex2_approx(m[half] - ref);  // 0 while nothing was visible
      m[half] = mn;
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = ex2_approx(y[i] - ref);
      l[half] = l[half] * scale[half] + ((e[0] + e[1]) + (e[2] + e[3]));
      // P in the cache's operand type for the second product, as in the other kernel; the sum is of the exact weights
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (kFp8) {
          const __half2 hp = __floats2half2_rn(e[2 * h], e[2 * h + 1]);
          pa[2 * h + half] = *reinterpret_cast<const uint32_t*>(&hp);
        } else {
          pa[2 * h + half] = pack_bf16x2(e[2 * h], e[2 * h + 1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      o[i][0] *= scale[0];
      o[i][1] *= scale[0];
      o[i][2] *= scale[1];
      o[i][3] *= scale[1];
      // column lane / 4 of product i is dim 16 (lane / 4) + i
      const uint32_t pick = (i & 1) ? 0x7632 : 0x5410;
      uint32_t b0, b1;
      asm("prmt.b32 %0, %1, %2, %3;" : "=r"(b0) : "r"(vw[0][i / 2]), "r"(vw[1][i / 2]), "r"(pick));
      asm("prmt.b32 %0, %1, %2, %3;" : "=r"(b1) : "r"(vw[2][i / 2]), "r"(vw[3][i / 2]), "r"(pick));
      mma<kFp8>(o[i], pa, b0, b1);
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    const int r = half ? r1 : r0;
    if (t == 0) {
      s_m[warp][r] = m[half];
      s_l[warp][r] = l[half];
    }
    // columns 2 t and 2 t + 1 of product i are dims 32 t + i and 32 t + 16 + i
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s_o[warp][r][32 * t + i] = o[i][2 * half];
      s_o[warp][r][32 * t + 16 + i] = o[i][2 * half + 1];
    }
  }
  __syncthreads();
  // the warps' states joined; every row sees its own node, so one of them holds something
  for (int i = tid; i < rows * (kHeadDim / 4); i += kThreads) {
    const int r = i % rows, quad = i / rows;
    float M = s_m[0][r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = ex2_approx(s_m[w][r] - M);
      const float* x = &s_o[w][r][4 * quad];
      L = fmaf(a, s_l[w][r], L);
      acc.x = fmaf(a, x[0], acc.x);
      acc.y = fmaf(a, x[1], acc.y);
      acc.z = fmaf(a, x[2], acc.z);
      acc.w = fmaf(a, x[3], acc.w);
    }
    __stcg(p.row_o(0, kvh, quad) + li0 + r, acc);
    if (quad == 0) {
      __stcg(p.row_ml(0, kvh) + li0 + r, make_float2(M, L));
      __stcg(p.row_at(0, kvh) + li0 + r, make_int4(kRowWhole | (page0 > 0 ? kRowShares : 0), 0, 0, 0));
    }
  }
}

}  // namespace small

cudaError_t launch_shared_small(const void* q, const void* k_cache, const void* v_cache, const SharedAttnParams& p,
                                bool fp8_cache, cudaStream_t stream) {
  const dim3 grid(p.hkv, p.batch);
  const auto* qb = static_cast<const __nv_bfloat16*>(q);
  return fp8_cache ? launch_pdl(small::small_kernel<true>, grid, dim3(small::kThreads), 0, stream, nullptr, qb, k_cache,
                                v_cache, p)
                   : launch_pdl(small::small_kernel<false>, grid, dim3(small::kThreads), 0, stream, nullptr, qb, k_cache,
                                v_cache, p);
}

}  // namespace jf
