// sample.cu -- jf_sample: one token per row of logits (sm_100a, SIMT + clusters).
//
// Design: a thread-block cluster takes a row.  While few rows are asked for, its CTAs hold the row in shared memory, so
// that each pass of the draw (sampling.cuh) is short; with many rows the barriers of wide clusters would dominate, and
// narrow clusters, down to one CTA a row, read the row again from L2 in each pass.  Measured on rows of 151936 float32
// entries with top-p alone (us; held in shared memory / read from memory, with the number of CTAs): 8 rows 33 (8) / 39
// (16); 32 rows 48 (4) / 58 (8); 64 rows 91 (4), 127 (8) / 90 (4); 128 rows 166 (4) / 151 (2).
#include "sampling.cuh"

namespace jf {
namespace smp {

template <typename T, bool kResident>
__global__ void __launch_bounds__(kThreads, 2)
    sample_kernel(const T* __restrict__ logits, long long row_stride, int vocab, const float* __restrict__ u,
                  const SampleParams sp, int32_t* __restrict__ token, float* __restrict__ logprob, int32_t* status) {
  extern __shared__ __align__(128) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const long long r = blockIdx.x / C;
  const int tid = threadIdx.x;
  Row<T, kResident> row(s, raw + kSliceOff, rank, C, vocab);
  cluster.sync();  // every CTA of the cluster runs (remote shared memory may be written); the barrier is initialised
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the logits come from the kernel before this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  row.start(logits + r * row_stride);
  if (tid == kThreads - 1) s.rp = read_params(sp, r, __ldg(u + r));
  const Drawn d = row.template draw<false>(0);
  if (!d.ok) {
    volatile int never = 0;
    mbar_wait(&s.bar, 0, &never);  // no copy of this CTA is left in flight
    if (rank == 0 && tid == 0) report(status, JF_ERR_TIMEOUT);
    return;
  }
  if (!s.rp.ok) {  // the same in every CTA of the cluster
    if (rank == 0 && tid == 0) report(status, JF_ERR_DEVICE_CHECK);
    return;
  }
  if (d.mine) {
    token[r] = d.token;
    if (logprob != nullptr) logprob[r] = d.logprob;
  }
}

template <typename T, bool kResident>
cudaError_t launch(int cluster, size_t smem, const T* logits, long long row_stride, int rows, int vocab, const float* u,
                   const SampleParams& sp, int32_t* token, float* logprob, int32_t* status, cudaStream_t stream) {
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = prepare_kernel(sample_kernel<T, kResident>, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  return launch_pdl(sample_kernel<T, kResident>, dim3(static_cast<unsigned>(rows) * cluster), dim3(kThreads), smem,
                    stream, &attr, logits, row_stride, vocab, u, sp, token, logprob, status);
}

template <typename T>
cudaError_t choose(const T* logits, long long row_stride, int rows, int vocab, const float* u, const SampleParams& sp,
                   int32_t* token, float* logprob, int32_t* status, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  int c = widest_cluster(rows, vocab, sms);
  const size_t smem = kSliceOff + slice_bytes(vocab, c, sizeof(T));
  if (smem <= (rows * static_cast<long long>(c) <= sms ? kMaxDynSmem : kTwoPerSm))
    return launch<T, true>(c, smem, logits, row_stride, rows, vocab, u, sp, token, logprob, status, stream);
  // Slices that do not fit: two CTAs an SM, and one CTA a row where two would be more than that.  Whether one is right
  // there depends on the filters, which lie on the device: a small top-k is a chain of dependent phases that a second
  // CTA only delays, while passes over the weights gain from it as long as SMs are left with a single row.  Small top-k
  // with top-p and min-p, no filter, top-p, mixed filters (us, one CTA a row / two), 150 float32 rows of 66001 entries:
  // 48 / 54, 48 / 45, 130 / 93, 129 / 92; 222 of them: 51 / 64, 50 / 47, 136 / 137, 148 / 120; 222 of 151936:
  // 103 / 112, 105 / 86, 276 / 260, 276 / 195.  No filter and top-p, 256 of 151936: 107 / 109, 280 / 276; 512:
  // 202 / 183, 501 / 487; 1024: 344 / 352, 906 / 889.
  while (c < kMaxCluster && rows * 2ll * c <= 2 * sms && slice_len(vocab, c) > kMinSlice) c *= 2;
  return launch<T, false>(c, kSliceOff, logits, row_stride, rows, vocab, u, sp, token, logprob, status, stream);
}

}  // namespace smp

#ifdef JF_DEBUG
cudaError_t hold_sample(int on) { return cudaMemcpyToSymbol(smp::g_hold, &on, sizeof(on)); }
#endif

cudaError_t launch_sample(const void* logits, bool bf16, long long row_stride, int rows, int vocab, const float* u,
                          const SampleParams& sp, int32_t* token, float* logprob, int32_t* status,
                          cudaStream_t stream) {
  return bf16 ? smp::choose(static_cast<const __nv_bfloat16*>(logits), row_stride, rows, vocab, u, sp, token, logprob,
                            status, stream)
              : smp::choose(static_cast<const float*>(logits), row_stride, rows, vocab, u, sp, token, logprob, status,
                            stream);
}

}  // namespace jf
