// out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the pieces s of a row, M = max_s m_s:
// the log-sum-exp join of partial softmax results (m_s the piece's running maximum in log2
// units, l_s its sum, o_s its unnormalised output). The statistics stay in fp32.
//
// Latency-bound: the pieces were just written and lie in L2, so what counts is the number of
// dependent rounds of loads. A thread takes four consecutive outputs and has the loads of up
// to six pieces in flight; a row of more pieces is shared by up to 64 threads per output, which
// join pairwise through shared memory. One request of 16000 positions in 150 pieces: 12.4 us the
// step, 19.7 with eight threads at most and two key warps' pieces of each CTA; 64 requests of 128 ..
// 2048 positions with four or eight pieces in flight: 31.9 and 31.6 us, 30.4 with six.
#include <float.h>

#include <algorithm>

#include "common.cuh"
#include "merge.h"

namespace cb {

namespace {

constexpr int kInFlight = 6;
constexpr int kMaxParts = 64;

struct Acc {
  float m, l;
  float4 o;
};

CB_DEV void join(Acc& x, float m, float l, float4 o) {
  const float M = fmaxf(x.m, m);
  const float a = exp2f(x.m - M), b = exp2f(m - M);
  x.m = M;
  x.l = x.l * a + l * b;
  x.o.x = x.o.x * a + o.x * b;
  x.o.y = x.o.y * a + o.y * b;
  x.o.z = x.o.z * a + o.z * b;
  x.o.w = x.o.w * a + o.w * b;
}

}  // namespace

// The rows travel in the kernel arguments, so that the merge waits for no copy: few of them in a
// small argument block (the copy of a large one costs a small step), many in few launches.
template <int N>
struct RowList {
  MergeRow rows[N];
};

template <typename T, int N>
__global__ void __launch_bounds__(kMergeThreads)
merge_rows_kernel(const MergeArgs m, const __grid_constant__ RowList<N> list) {
  __shared__ float4 sh_o[kMergeThreads];
  __shared__ float2 sh_ml[kMergeThreads];
  const MergeRow& row = list.rows[blockIdx.x];
  const int per = kMergeThreads / m.parts;  // outputs (of four values) per CTA
  const int part = threadIdx.x / per;
  const int f = blockIdx.y * per + threadIdx.x % per;
  const int F = m.num_q_heads * m.head_dim / 4;
  const int h = f * 4 / m.head_dim;
  const int n = row.na + row.nb;
  allow_dependent_launch();
  grid_dependency_wait();
  Acc x{-FLT_MAX, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (f < F) {
    const float4* o = reinterpret_cast<const float4*>(m.part_o);
    const int s1 = (part + 1) * n / m.parts;
    for (int s0 = part * n / m.parts; s0 < s1; s0 += kInFlight) {
      float2 ml[kInFlight];
      float4 v[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int s = s0 + i;
        if (s < s1) {
          const long long pr = s < row.na ? (long long)row.a + (long long)s * row.a_step
                                          : (long long)row.b + (long long)(s - row.na) * row.b_step;
          ml[i] = __ldcg(m.part_ml + pr * m.num_q_heads + h);
          v[i] = __ldcg(o + pr * F + f);
        }
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i)
        if (s0 + i < s1) join(x, ml[i].x, ml[i].y, v[i]);
    }
  }
  if (m.parts > 1) {
    sh_o[threadIdx.x] = x.o;
    sh_ml[threadIdx.x] = make_float2(x.m, x.l);
    for (int half = m.parts / 2; half > 0; half /= 2) {  // parts and kMergeThreads are powers of two
      __syncthreads();
      if (part < half) {
        const int other = threadIdx.x + half * per;
        join(x, sh_ml[other].x, sh_ml[other].y, sh_o[other]);
        sh_o[threadIdx.x] = x.o;
        sh_ml[threadIdx.x] = make_float2(x.m, x.l);
      }
    }
  }
  if (part != 0 || f >= F) return;
  const float inv = x.l != 0.f ? 1.f / x.l : 0.f;
  T* out = static_cast<T*>(m.out) + (long long)row.t * F * 4 + 4 * f;
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(out) = make_float4(x.o.x * inv, x.o.y * inv, x.o.z * inv, x.o.w * inv);
  } else {
    __nv_bfloat162 a = __floats2bfloat162_rn(x.o.x * inv, x.o.y * inv);
    __nv_bfloat162 b = __floats2bfloat162_rn(x.o.z * inv, x.o.w * inv);
    *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
  }
}

int merge_parts(int pieces) {
  int parts = 1;
  while (parts < kMaxParts && pieces > kInFlight * parts) parts *= 2;
  return parts;
}

namespace {

template <int N>
cudaError_t launch_rows(const MergeArgs& m, const MergeRow* rows, int n, cudaStream_t stream) {
  const int per = kMergeThreads / m.parts;
  const int F = m.num_q_heads * m.head_dim / 4;
  for (int i = 0; i < n; i += N) {
    const int k = std::min(N, n - i);
    RowList<N> list;
    std::copy(rows + i, rows + i + k, list.rows);
    const dim3 grid(k, (F + per - 1) / per);
    const cudaError_t e =
        m.dtype == 0
            ? launch_pdl(kMergeRowsId, merge_rows_kernel<float, N>, grid, dim3(kMergeThreads), 0, stream, m, list)
            : launch_pdl(kMergeRowsId, merge_rows_kernel<__nv_bfloat16, N>, grid, dim3(kMergeThreads), 0, stream, m, list);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_merge(const MergeArgs& m, const MergeRow* rows, int n, cudaStream_t stream) {
  if (n <= 64) return launch_rows<64>(m, rows, n, stream);
  return launch_rows<1024>(m, rows, n, stream);
}

}  // namespace cb
