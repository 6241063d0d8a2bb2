// sample.cu -- jf_sample: one token per row of logits (sm_100a, SIMT + clusters).
//
// Design: one thread-block cluster per row.  The row is read from memory once, by bulk copies into the shared memory
// of the cluster's CTAs, and every pass of the draw (sampling.cuh) then reads it there.
#include "sampling.cuh"

namespace jf {
namespace smp {

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    sample_kernel(const T* __restrict__ logits, long long row_stride, int vocab, const float* __restrict__ u,
                  const SampleParams sp, int32_t* __restrict__ token, float* __restrict__ logprob, int32_t* status) {
  extern __shared__ __align__(128) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const long long r = blockIdx.x / C;
  const int tid = threadIdx.x;
  Row<T> row(s, raw + kSliceOff, rank, C, vocab);
  cluster.sync();  // every CTA of the cluster runs (remote shared memory may be written); the barrier is initialised
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the logits come from the kernel before this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  RowParams rp;
  const float ur = __ldg(u + r);
  if (!read_params(sp, r, rp) || !good_u(ur)) {  // the same in every CTA of the cluster
    if (rank == 0 && tid == 0) report(status, JF_ERR_DEVICE_CHECK);
    return;
  }
  row.start(logits + r * row_stride);
  const Drawn d = row.template draw<false>(rp, ur, 0);
  if (!d.ok) {
    volatile int never = 0;
    mbar_wait(&s.bar, 0, &never);  // no copy of this CTA is left in flight
    if (rank == 0 && tid == 0) report(status, JF_ERR_TIMEOUT);
    return;
  }
  if (d.mine) {
    token[r] = d.token;
    if (logprob != nullptr) logprob[r] = d.logprob;
  }
}

template <typename T>
cudaError_t launch(const T* logits, long long row_stride, int rows, int vocab, const float* u, const SampleParams& sp,
                   int32_t* token, float* logprob, int32_t* status, cudaStream_t stream) {
  static std::atomic<int> sms_of[kMaxDevices];
  const int sms = prepare_kernel(sample_kernel<T>, sms_of);
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int cluster = cluster_size(rows, vocab, sizeof(T), sms);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  return launch_pdl(sample_kernel<T>, dim3(static_cast<unsigned>(rows) * cluster), dim3(kThreads),
                    kSliceOff + slice_bytes(vocab, cluster, sizeof(T)), stream, &attr, logits, row_stride, vocab, u, sp,
                    token, logprob, status);
}

}  // namespace smp

cudaError_t launch_sample(const void* logits, bool bf16, long long row_stride, int rows, int vocab, const float* u,
                          const SampleParams& sp, int32_t* token, float* logprob, int32_t* status,
                          cudaStream_t stream) {
  return bf16 ? smp::launch(static_cast<const __nv_bfloat16*>(logits), row_stride, rows, vocab, u, sp, token, logprob,
                            status, stream)
              : smp::launch(static_cast<const float*>(logits), row_stride, rows, vocab, u, sp, token, logprob, status,
                            stream);
}

}  // namespace jf
