// topk_lens.cu -- the decode selection for a batch whose sequences have
// their own lengths: row r of the scores belongs to sequence r / rows_per_len,
// which has n = ceil(len / block) blocks; candidates are the blocks j < n-1,
// the sequence's last block n-1 is always kept (SAS page, 推理 paragraph and
// 核心模块 3; "稀疏注意力" tutorial §5), and columns past it are not read: in a
// growing cache they hold whatever was there before.
#include "kernels.h"
#include "topk.cuh"

namespace bsa {
namespace topk_lens {

template <int KPT>
__global__ void __launch_bounds__(256) cta_kernel(const float* __restrict__ scores, int ncols,
                                                  const int* __restrict__ lens, int rows_per_len, int block, int kb,
                                                  int* __restrict__ idx_out, int idx_stride,
                                                  int* __restrict__ count_out, uint32_t* __restrict__ status) {
  griddep_wait();   // the scores come from the kernel launched before
  const int64_t r = blockIdx.x;
  const int len = lens[r / rows_per_len];
  const int n_all = len > 0 ? (len - 1) / block + 1 : 0;
  if (n_all > ncols && threadIdx.x == 0) atomicOr(status, BSA_DEV_BAD_INDEX);
  const int n = min(n_all, ncols);
  const int ncand = max(n - 1, 0);
  const float* srow = scores + r * ncols;
  const int j0 = threadIdx.x * KPT;
  uint32_t key[KPT];
#pragma unroll
  for (int e = 0; e < KPT; ++e) key[e] = (j0 + e < ncand) ? order_key(__ldg(srow + j0 + e)) : 0u;
  cta_topk_select<KPT>(key, ncand, kb, n - 1, idx_out + r * idx_stride, idx_stride,
                       count_out ? count_out + r : nullptr);
}

}  // namespace topk_lens

cudaError_t launch_topk_lens(const float* scores, int rows, int ncols, const int* lens, int rows_per_len, int block,
                             int kb, int* idx_out, int idx_stride, int* count_out, uint32_t* status,
                             cudaStream_t st) {
  auto kernel = ncols <= 256 * 2 ? topk_lens::cta_kernel<2>
                                 : (ncols <= 256 * 8 ? topk_lens::cta_kernel<8> : topk_lens::cta_kernel<32>);
  return launch_dependent(kernel, dim3(rows), dim3(256), 0, st, scores, ncols, lens, rows_per_len, block, kb, idx_out,
                          idx_stride, count_out, status);
}

}  // namespace bsa
