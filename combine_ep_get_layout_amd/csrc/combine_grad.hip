// Gradient of combine on gfx950.  out[t] = sum_k w[t][k] y[row(t, k)], so
//   dy[row(t, k)] = w[t][k] dout[t]     and     dw[t][k] = <dout[t], y[row(t, k)]>;
// in rank-major mode out[t] is the unweighted sum of the token's distinct
// rows, so dy[row] = dout[t].
//
// One workgroup per token: dout[t] comes from memory once, then each
// routed row is read (y) and written (dy) as one stream.  Bound by memory:
// the rows read and written are all but 1 / (2 K) of its bytes.  262,144 rows x 7168:
// 1.58 ms, 5.0 TB/s, 92% of a plain copy's rate.  All eight rows of a token in
// flight at once, in workgroups of 64 to 448 threads, take the same 1.585 to
// 1.595 ms, and a small case 6.3 us instead of 4.0.
#include "ep_device.hpp"
#include "ep_internal.hpp"

namespace ep {

__device__ __forceinline__ uint32_t bf16_any(float f) {
  return f != f ? ((__float_as_uint(f) >> 16) | 0x40u) : f32_to_bf16_rne(f);
}

constexpr int kGradThreads = 256;

template <bool RM>
__global__ __launch_bounds__(kGradThreads) void combine_grad(CombineGradArgs a, int64_t first) {
  __shared__ float part[64][kGradThreads / kWave];
  const int V = a.g.H / 8, K = a.g.K;
  const int64_t tok = first + blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int myrow = lane < K ? a.send_pos[tok * K + lane] : -1;
  const float myw = !RM && lane < K && a.w ? a.w[tok * K + lane] : 1.0f;
  if (__ballot(myrow >= a.rows) != 0 && threadIdx.x == 0) set_err(a.err, EP_DEVERR_CAPACITY);
  const u32x4* dout = (const u32x4*)a.dout + tok * V;
  for (int k = 0; k < K; ++k) {
    const int row = __builtin_amdgcn_readlane(myrow, k);
    float dot = 0.0f;
    bool again = false;  // rank-major: an earlier entry's row
    if (RM)
      for (int q = 0; q < k; ++q) again |= __builtin_amdgcn_readlane(myrow, q) == row;
    if (row >= 0 && row < a.rows && !again) {
      const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(myw), k));
      for (int j = threadIdx.x; j < V; j += kGradThreads) {
        const u32x4 d = dout[j];
        if (a.dw) {
          const u32x4 y = __builtin_nontemporal_load((const u32x4*)a.y + (int64_t)row * V + j);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            dot = __builtin_fmaf(bf16_lo(d[q]), bf16_lo(y[q]), dot);
            dot = __builtin_fmaf(bf16_hi(d[q]), bf16_hi(y[q]), dot);
          }
        }
        if (a.dy) {
          u32x4 o = d;
          if (!RM)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              o[q] = bf16_any(w * bf16_lo(d[q])) | (bf16_any(w * bf16_hi(d[q])) << 16);
          __builtin_nontemporal_store(o, (u32x4*)a.dy + (int64_t)row * V + j);
        }
      }
    }
    if (a.dw) {
#pragma unroll
      for (int s = 32; s > 0; s >>= 1) dot += __shfl_xor(dot, s);
      if (lane == 0) part[k][wave] = dot;
    }
  }
  if (a.dw) {
    __syncthreads();
    if ((int)threadIdx.x < K) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < kGradThreads / kWave; ++q) s += part[threadIdx.x][q];
      a.dw[tok * K + threadIdx.x] = s;
    }
  }
}

// Tokens of a launch: a grid holds fewer than 2^32 threads.
constexpr int64_t kGradTokens = (1ll << 31) / kGradThreads;

hipError_t launch_combine_grad(const CombineGradArgs& a, hipStream_t st) {
  const int64_t N = (int64_t)a.g.R * a.g.T;
  for (int64_t first = 0; first < N; first += kGradTokens) {
    const dim3 grid((unsigned)(N - first < kGradTokens ? N - first : kGradTokens));
    if (a.rank_major)
      hipLaunchKernelGGL(combine_grad<true>, grid, dim3(kGradThreads), 0, st, a, first);
    else
      hipLaunchKernelGGL(combine_grad<false>, grid, dim3(kGradThreads), 0, st, a, first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace ep
