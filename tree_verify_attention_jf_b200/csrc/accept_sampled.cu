// accept_sampled.cu -- jf_accept_sampled: the acceptance walk over the verified draft tree with a sampled token in
// place of the target's argmax (sm_100a, SIMT + clusters).
//
// Design: the walk is a chain of dependent draws, so latency matters.  One cluster per sequence; each step brings the
// current node's row into the cluster's shared memory and draws from it (sampling.cuh); every CTA knows the token drawn
// and finds the same child in its own copy of the tree.  While a row is drawn from, the rows of the node's first
// children, the only candidates for the next step, are prefetched into L2.  Measured: a step of one sequence takes
// about 10 us (151936 entries, top-k, top-p and min-p), of 8 sequences with nucleus sampling 21 us.
#include "sampling.cuh"

namespace jf {
namespace smp {

struct Tree {
  int tok[kMaxAcceptNodes], par[kMaxAcceptNodes];
  int kid[2];  // the child found, by step parity
  int ahead;   // rows prefetched in this step
};
constexpr int kAhead = 8;  // a tree's nodes rarely have more children than the eight candidates they are built from
// Bytes prefetched in a step by the whole batch, a small part of the L2: rows that are not used push out what is (us,
// without a bound / with this one / none prefetched, 151936 entries: 8 float32 sequences with top-p 236 / 233 / 230, 40
// of them 332 / 326 / 326, one 62 / 62 / 62; 4 bf16 ones whose rows lie in HBM alone 163 / 163 / 165).
constexpr size_t kAheadBytes = 20 << 20;
constexpr size_t kTreeOff = kSliceOff;
constexpr size_t kWalkSliceOff = (kTreeOff + sizeof(Tree) + 127) & ~size_t(127);

template <typename T>
__global__ void __launch_bounds__(kThreads)
    accept_sampled_kernel(const int32_t* __restrict__ token, const int32_t* __restrict__ parent,
                          const T* __restrict__ logits, const float* __restrict__ u, const SampleParams sp,
                          int num_nodes, int vocab, int max_depth, int ahead, int32_t* __restrict__ accepted_len,
                          int32_t* __restrict__ path, int32_t* __restrict__ bonus, float* __restrict__ logprob,
                          int32_t* status) {
  extern __shared__ __align__(128) uint8_t raw[];
  __shared__ int s_path[kMaxAcceptNodes + 1];
  __shared__ float s_lp[kMaxAcceptNodes];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  Tree& t = *reinterpret_cast<Tree*>(raw + kTreeOff);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const long long b = blockIdx.x / C;
  const int tid = threadIdx.x;
  Row<T, true> row(s, raw + kWalkSliceOff, rank, C, vocab);
  cluster.sync();  // every CTA of the cluster runs (remote shared memory may be written); the barrier is initialised
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before this one has completed
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const T* rows = logits + b * num_nodes * vocab;
  const float* ub = u + b * (max_depth + 1);
  bool bad = false;
  for (int i = tid; i < num_nodes; i += kThreads) {
    const int pi = __ldg(parent + b * num_nodes + i);
    t.par[i] = pi;
    t.tok[i] = __ldg(token + b * num_nodes + i);
    bad = bad || pi < -1 || pi >= i;
  }
  if (tid == kThreads - 1) s.rp = read_params(sp, b, 0.f);
  bad = __syncthreads_or(bad) || !s.rp.ok;  // the same in every CTA of the cluster
  if (bad) {
    if (rank == 0 && tid == 0) report(status, JF_ERR_DEVICE_CHECK);
    return;
  }
  int cur = 0, L = 0, drawn = -1;
  for (int step = 0;; ++step) {
    const float us = __ldg(ub + step);  // step == L <= max_depth
    if (!s.rp.greedy && !(us >= 0.f && us < 1.f)) {
      if (rank == 0 && tid == 0) report(status, JF_ERR_DEVICE_CHECK);
      return;  // between two draws no CTA writes into another's shared memory
    }
    if (tid == 0) {
      s.rp.u = us;
      t.kid[step & 1] = INT_MAX;
      t.ahead = 0;
    }
    fence_proxy_async_smem();
    __syncthreads();  // the previous row's last reads are done before the copy of this one starts
    row.start(rows + static_cast<long long>(cur) * vocab);
    if (L < max_depth && ahead > 0)
      for (int c = tid; c < num_nodes; c += kThreads)
        if (t.par[c] == cur && atomicAdd(&t.ahead, 1) < ahead) row.prefetch(rows + static_cast<long long>(c) * vocab);
    const Drawn d = row.template draw<true>(step & 1);
    if (!d.ok) {
      volatile int never = 0;
      mbar_wait(&s.bar, step & 1, &never);  // no copy of this CTA is left in flight
      if (rank == 0 && tid == 0) report(status, JF_ERR_TIMEOUT);
      return;
    }
    drawn = d.token;
    if (tid == 0) {
      s_path[L] = cur;
      s_lp[L] = d.logprob;
    }
    if (L == max_depth || drawn < 0) break;
    for (int c = tid; c < num_nodes; c += kThreads)
      if (t.par[c] == cur && t.tok[c] == drawn) atomicMin(&t.kid[step & 1], c);
    __syncthreads();
    const int kid = t.kid[step & 1];
    if (kid == INT_MAX) break;
    cur = kid;
    ++L;
  }
  if (rank != 0) return;
  __syncthreads();
  if (tid == 0) {
    accepted_len[b] = L;
    bonus[b] = drawn;
  }
  for (int i = tid; i <= max_depth; i += kThreads) {
    path[b * (max_depth + 1) + i] = i <= L ? s_path[i] : -1;
    if (logprob != nullptr) logprob[b * (max_depth + 1) + i] = i <= L ? s_lp[i] : 0.f;
  }
}

template <typename T>
cudaError_t launch_walk(int cluster, size_t smem, const int32_t* token, const int32_t* parent, const T* logits,
                        const float* u, const SampleParams& sp, int batch, int num_nodes, int vocab, int max_depth,
                        int32_t* accepted_len, int32_t* path, int32_t* bonus, float* logprob, int32_t* status,
                        cudaStream_t stream) {
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = prepare_kernel(accept_sampled_kernel<T>, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  const size_t rows_ahead = kAheadBytes / (static_cast<size_t>(batch) * vocab * sizeof(T));
  const int ahead = static_cast<int>(rows_ahead < kAhead ? rows_ahead : kAhead);
  return launch_pdl(accept_sampled_kernel<T>, dim3(static_cast<unsigned>(batch) * cluster), dim3(kThreads), smem,
                    stream, &attr, token, parent, logits, u, sp, num_nodes, vocab, max_depth, ahead, accepted_len,
                    path, bonus, logprob, status);
}

// The cluster is as wide as its row's slices need to fit shared memory, if that is wider than the rule for all
// sequences at once: clusters then wait for SMs, which costs less than reading rows from memory in every pass of a
// draw.  Measured on 151936 float32 entries with top-p, four steps (us; slices in shared memory / one narrow cluster a
// sequence and rows read from memory): 38 sequences 224 / 444, 74: 342 / 478, 150: 556 / 932, 300: 1030 / 1560; 80
// sequences with rows of 45001 entries 166 / 279, of 524288 1305 / 4624.
static_assert(kWalkSliceOff + slice_bytes(kMaxSampleVocab, kMaxCluster, sizeof(float)) <= kMaxDynSmem,
              "the widest cluster holds any row");
template <typename T>
cudaError_t choose_walk(const int32_t* token, const int32_t* parent, const T* logits, const float* u,
                        const SampleParams& sp, int batch, int num_nodes, int vocab, int max_depth,
                        int32_t* accepted_len, int32_t* path, int32_t* bonus, float* logprob, int32_t* status,
                        cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  int c = widest_cluster(batch, vocab, sms);
  while (kWalkSliceOff + slice_bytes(vocab, c, sizeof(T)) > kMaxDynSmem) c *= 2;
  return launch_walk<T>(c, kWalkSliceOff + slice_bytes(vocab, c, sizeof(T)), token, parent, logits, u, sp, batch,
                        num_nodes, vocab, max_depth, accepted_len, path, bonus, logprob, status, stream);
}

}  // namespace smp

#ifdef JF_DEBUG
cudaError_t hold_accept_sampled(int on) { return cudaMemcpyToSymbol(smp::g_hold, &on, sizeof(on)); }
#endif

cudaError_t launch_accept_sampled(const int32_t* token, const int32_t* parent, const void* logits, bool bf16,
                                  const float* u, const SampleParams& sp, int batch, int num_nodes, int vocab,
                                  int max_depth, int32_t* accepted_len, int32_t* path, int32_t* bonus, float* logprob,
                                  int32_t* status, cudaStream_t stream) {
  return bf16 ? smp::choose_walk(token, parent, static_cast<const __nv_bfloat16*>(logits), u, sp, batch, num_nodes,
                                 vocab, max_depth, accepted_len, path, bonus, logprob, status, stream)
              : smp::choose_walk(token, parent, static_cast<const float*>(logits), u, sp, batch, num_nodes, vocab,
                                 max_depth, accepted_len, path, bonus, logprob, status, stream);
}

}  // namespace jf
