// topk_lens.cu -- the decode selection for a batch whose sequences have
// their own lengths: row r of the scores belongs to sequence r / rows_per_len,
// which has n = ceil(len / block) blocks; candidates are the blocks j < n-1,
// the sequence's last block n-1 is always kept (SAS page, 推理 paragraph and
// 核心模块 3; "稀疏注意力" tutorial §5), and columns from it on do not count: in a
// growing cache they hold whatever was there before.
//
// One warp per row (four past 2048 columns, whose counts meet in shared memory),
// the row's scores in its registers as bf16 pairs (rounded to nearest, which
// keeps their order up to ties).  A row is a few KB, so
// instructions count, not bytes: the bf16 threshold T (the largest with at
// least k scores >= T) is found by bisection of the 16-bit codes, 16 counts at
// one compare and one add for two scores.
// Scores whose rounding is above T are kept; those that round to T (a few,
// as a rule) are listed and ranked by their full keys, or, where more than 32
// do, their lower key bits are bisected by 32 more counts over the row.
// Equal scores: the lower index first.  NaN compares with nothing, so it ranks
// last by itself.  The counts run over registers; then each lane takes 64
// consecutive columns (32 or 16 in short rows) from shared memory, keeps what is
// above T and what rounds to it as bits, and writes its kept columns behind
// those of the lanes before it: no step waits for another column's.  2048 rows
// of 1300 candidates: 11.5 us; a block of 256 threads a row with four 8-bit
// histograms took 21.2, one 12-bit histogram and a ranked list 22.3, ballots
// column by column instead of the lanes' bits 13.9.
#include "kernels.h"
#include "topk.cuh"

namespace bsa {
namespace topk_lens {

__device__ __forceinline__ __nv_bfloat162 as_pair(uint32_t v) { return *reinterpret_cast<__nv_bfloat162*>(&v); }
// A 16-bit code that orders as the bf16 values do, and back.
__device__ __forceinline__ uint32_t code_value(uint32_t code) { return code & 0x8000u ? code & 0x7FFFu : ~code & 0xFFFFu; }

// Sums over a row's warps, and what stands in the warps before; every warp calls them in step.  Two places in
// turn: a warp may write the next sum while another still reads this one.
template <int WARPS>
struct Across {
  int* place;       // [2][WARPS], shared
  int turn = 0;
  __device__ __forceinline__ explicit Across(int* shared) : place(shared) {}
  __device__ __forceinline__ int sum(int v) {
    int before;
    return sum(v, before);
  }
  __device__ __forceinline__ int sum(int v, int& before) {
    before = 0;
    if constexpr (WARPS > 1) {
      const int warp = threadIdx.x >> 5;
      int* at = place + turn * WARPS;
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) at[warp] = v;
      __syncthreads();
      v = 0;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) {
        if (k < warp) before += at[k];
        v += at[k];
      }
    }
    return v;
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    if constexpr (WARPS > 1) {
      uint32_t* at = reinterpret_cast<uint32_t*>(place) + turn * WARPS;
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = v;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < WARPS; ++k) v = ::max(v, at[k]);
    }
    return v;
  }
};

template <int PAIRS>
__device__ __forceinline__ int count_ge(const uint32_t (&x)[PAIRS], uint32_t code) {
  const uint32_t t = code_value(code);
  const uint32_t both = t | (t << 16);
  __nv_bfloat162 acc[4];       // at most 256 each: exact in bf16
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = __hge2(as_pair(x[i]), as_pair(both));
#pragma unroll
  for (int p = 4; p < PAIRS; ++p) acc[p & 3] = __hadd2(acc[p & 3], __hge2(as_pair(x[p]), as_pair(both)));
  float c = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(acc[i]);
    c += f.x + f.y;
  }
  return __reduce_add_sync(0xffffffffu, static_cast<int>(c));
}

// Code of the row's largest score, below every number's where all are NaN.
template <int PAIRS>
__device__ __forceinline__ uint32_t code_max(const uint32_t (&x)[PAIRS]) {
  __nv_bfloat162 m = as_pair(x[0]);
#pragma unroll
  for (int p = 1; p < PAIRS; ++p) m = __hmax2(m, as_pair(x[p]));       // the other one, where one is NaN
  const uint32_t bits = *reinterpret_cast<const uint32_t*>(&m);
  uint32_t best = 0u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t v = (bits >> (16 * h)) & 0xFFFFu;
    const bool is_nan = (v & 0x7FFFu) > 0x7F80u;
    const uint32_t code = v & 0x8000u ? ~v & 0xFFFFu : v | 0x8000u;
    best = max(best, is_nan ? 0u : code);
  }
  return __reduce_max_sync(0xffffffffu, best);
}

// Pair p of lane l of warp w holds columns 64 (PAIRS w + p) + 2 l and the next one.
template <int PAIRS, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) row_kernel(const float* __restrict__ scores, int ncols,
                                                 const int* __restrict__ lens, int rows_per_len, int block, int kb,
                                                 int* __restrict__ idx_out, int idx_stride,
                                                 int* __restrict__ count_out, uint32_t* __restrict__ status) {
  griddep_wait();   // the scores come from the kernel launched before
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col0 = warp * PAIRS * 64;                       // first column of this warp
  const int64_t r = blockIdx.x;
  const int len = lens[r / rows_per_len];
  const int n_all = len > 0 ? (len - 1) / block + 1 : 0;
  if (n_all > ncols && threadIdx.x == 0) atomicOr(status, BSA_DEV_BAD_INDEX);
  const int n = min(n_all, ncols);
  const int ncand = max(n - 1, 0);
  const float* srow = scores + r * ncols;
  const float nan = __uint_as_float(0x7FFFFFFFu);
  // a gap behind each lane's pairs keeps the lanes' banks apart
  __shared__ float2 xs_all[WARPS][PAIRS * 32 + 32];
  __shared__ uint32_t member_key[32];
  __shared__ int sums[2 * WARPS];
  float2* xs = xs_all[warp];
  Across<WARPS> across(sums);
  auto slot = [](int pair) { return pair + pair / PAIRS; };
  uint32_t x[PAIRS];
  // asked for together: no branch stands between the loads
  const bool even = ncols % 2 == 0 && (reinterpret_cast<uintptr_t>(scores) & 7u) == 0;
  {
    float2 v[PAIRS];
    if (even) {
#pragma unroll
      for (int p = 0; p < PAIRS; ++p) {
        const int j = col0 + 64 * p + 2 * lane;
        v[p] = j < ncand ? __ldg(reinterpret_cast<const float2*>(srow + j)) : make_float2(nan, nan);
      }
    } else {
#pragma unroll
      for (int p = 0; p < PAIRS; ++p) {
        const int j = col0 + 64 * p + 2 * lane;
        v[p].x = j < ncand ? __ldg(srow + j) : nan;
        v[p].y = j + 1 < ncand ? __ldg(srow + j + 1) : nan;
      }
    }
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) {
      if (col0 + 64 * p + 2 * lane + 1 >= ncand) v[p].y = nan;     // the row's next column, where it was read
      x[p] = pack_bf16x2(v[p].x, v[p].y);
      xs[slot(32 * p + lane)] = v[p];
    }
  }
  const int take = min(kb, ncand);
  // kept: scores that round above T; of those that round to T, full keys above `thresh`; of the keys equal to it the
  // first `ties`.  Code kNone stands below every number's: there the scores that "round to T" are the NaNs.
  constexpr uint32_t kNone = 0x007Eu;
  uint32_t t_code = 0xFFFFu, thresh = 0u;     // nothing is kept
  int ties = 0, remaining = 0, members = 0;
  if (take > 0) {
    uint32_t lo = kNone, hi = max(across.max(code_max(x)), kNone);
    int at_least = ncand, above = 0;           // scores >= lo, > hi
    // the best scores lie in the octaves below the largest: 4 of them (128 codes each) are tried first, then 32
    uint32_t reach = 512u;
    while (lo < hi && at_least != take) {
      uint32_t mid = (lo + hi + 1) / 2;
      if (reach != 0u) {
        mid = hi > lo + reach ? hi - reach : mid;
        reach = reach == 512u ? 4096u : 0u;
      }
      const int c = across.sum(count_ge(x, mid));
      if (c >= take) {
        lo = mid;
        at_least = c;
        reach = 0u;
      } else {
        hi = mid - 1;
        above = c;
      }
    }
    t_code = lo;
    remaining = take - above;
    members = at_least - above;
    if (lo == kNone) ties = remaining;        // every number, and NaNs (key 0) in index order
  }
  // this lane's columns, 2 PAIRS consecutive ones: bits of those that round above T, and to T
  __syncwarp();
  const __nv_bfloat162 t2 = as_pair(code_value(t_code) * 0x10001u);
  const int pair0 = lane * PAIRS, lane_col0 = col0 + 2 * pair0;
  uint64_t gt = 0u, eq = 0u;
  const int left = ncand - lane_col0;                // its candidates
  if (left > 0 && take > 0) {
#pragma unroll 8
    for (int i = 0; i < PAIRS; ++i) {
      const float2 f = xs[slot(pair0 + i)];
      const __nv_bfloat162 v = as_pair(pack_bf16x2(f.x, f.y));
      uint32_t above_t, at_t;
      if (t_code == kNone) {
        above_t = __heq2_mask(v, v);
        at_t = ~above_t;
      } else {
        above_t = __hgt2_mask(v, t2);
        at_t = __heq2_mask(v, t2);
      }
      // a half of the mask is all ones or zeros: bits 0 and 31 tell
      gt |= static_cast<uint64_t>((above_t & 1u) | (above_t >> 31 << 1)) << (2 * i);
      eq |= static_cast<uint64_t>((at_t & 1u) | (at_t >> 31 << 1)) << (2 * i);
    }
    if (left < 64) {
      const uint64_t own = (1ull << left) - 1ull;
      gt &= own;
      eq &= own;
    }
  }
  auto key_at = [&](int bit) {
    const float2 f = xs[slot(pair0 + (bit >> 1))];
    return order_key(bit & 1 ? f.y : f.x);
  };
  // how many of the lanes and warps before, and of all
  auto count_before = [&](int mine, int& before) {
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int warps_before;
    const int all = across.sum(__shfl_sync(0xffffffffu, incl, 31), warps_before);
    before = warps_before + incl - mine;
    return all;
  };
  if (t_code != kNone && remaining < members) {
    if (members <= 32) {
      // the members' full keys in a list, each ranked against all
      int at;
      count_before(__popcll(eq), at);
      for (uint64_t m = eq; m; m &= m - 1) member_key[at++] = key_at(__ffsll(m) - 1);
      if constexpr (WARPS > 1) __syncthreads(); else __syncwarp();
      const uint32_t mine = lane < members ? member_key[lane] : 0u;
      int more = 0, same = 0;
      for (int i = 0; i < members; ++i) {
        const uint32_t other = member_key[i];
        more += other > mine ? 1 : 0;
        same += other == mine ? 1 : 0;
      }
      const bool is_it = lane < members && more < remaining && remaining <= more + same;
      const int src = __ffs(__ballot_sync(0xffffffffu, is_it)) - 1;
      thresh = __shfl_sync(0xffffffffu, mine, src);
      ties = remaining - __shfl_sync(0xffffffffu, more, src);
    } else {
      // many scores round to T: bisect their full keys
      int over = 0;
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t cand = thresh | (1u << bit);
        int c = 0;
        for (uint64_t m = eq; m; m &= m - 1) c += key_at(__ffsll(m) - 1) >= cand ? 1 : 0;
        if (across.sum(__reduce_add_sync(0xffffffffu, c)) >= remaining) thresh = cand;
      }
      for (uint64_t m = eq; m; m &= m - 1) over += key_at(__ffsll(m) - 1) > thresh ? 1 : 0;
      ties = remaining - across.sum(__reduce_add_sync(0xffffffffu, over));
    }
  }
  uint64_t sel = gt, tie = 0u;
  if (remaining > 0) {      // the same for the whole row
    for (uint64_t m = eq; m; m &= m - 1) {
      const uint32_t key = key_at(__ffsll(m) - 1);
      const uint64_t bit = m & (0ull - m);
      if (key > thresh) sel |= bit;
      if (key == thresh) tie |= bit;
    }
    // ties in index order: the first of those not yet taken by columns before this lane's
    int before;
    count_before(__popcll(tie), before);
    for (; tie != 0u && before < ties; tie &= tie - 1, ++before) sel |= tie & (0ull - tie);
  }
  int* out = idx_out + r * idx_stride;
  int at;
  int kept = count_before(__popcll(sel), at);
  for (; sel; sel &= sel - 1) out[at++] = lane_col0 + __ffsll(sel) - 1;
  if (n > 0) {
    if (threadIdx.x == 0) out[kept] = n - 1;
    ++kept;
  }
  for (int t = kept + threadIdx.x; t < idx_stride; t += 32 * WARPS) out[t] = -1;
  if (count_out && threadIdx.x == 0) count_out[r] = kept;
}

}  // namespace topk_lens

cudaError_t launch_topk_lens(const float* scores, int rows, int ncols, const int* lens, int rows_per_len, int block,
                             int kb, int* idx_out, int idx_stride, int* count_out, uint32_t* status,
                             cudaStream_t st) {
  // A warp for up to 2048 columns, four for more (us: 2048 rows of up to 8000 columns 33.0, by one warp 44.3; of 2048
  // columns 11.6 by one warp, 13.0 by two, 15.8 by four); no wider than the row needs: a lane writes its columns one by
  // one (2048 rows of up to 700 blocks 14.5 with 64 columns a lane, 9.5 with 32).
  if (ncols > 64 * 32)
    return launch_dependent(topk_lens::row_kernel<32, 4>, dim3(rows), dim3(128), 0, st, scores, ncols, lens, rows_per_len,
                            block, kb, idx_out, idx_stride, count_out, status);
  auto kernel = ncols <= 64 * 8 ? topk_lens::row_kernel<8, 1>
                                : (ncols <= 64 * 16 ? topk_lens::row_kernel<16, 1> : topk_lens::row_kernel<32, 1>);
  return launch_dependent(kernel, dim3(rows), dim3(32), 0, st, scores, ncols, lens, rows_per_len, block, kb, idx_out,
                          idx_stride, count_out, status);
}

}  // namespace bsa
