// Causal attention of a chunk of new tokens over the KV cache (include/mfa.h:
// mfa_chunk_attn).
//
// out[t][h] = sum_{j <= p_t} softmax_j(scale q[t][h] . K[j]) V[j], with the running maximum
// and sum of the softmax in float32. One warp per (token, head): a lane holds eight of the
// 256 dimensions, every key costs one warp-wide sum.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "mfa_internal.cuh"
#include "sm100.cuh"

namespace mfa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void load8(const KvSeq& s, const void* base, int dtype, long long at,
                                      int lane, float (&f)[8]) {
  if (dtype == MFA_KV_BF16) {
    const uint4 v =
        *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at * kHeadDim + 8 * lane);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const uint2 v =
        *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + at * kHeadDim + 8 * lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = i < 4 ? v.x : v.y;
      __nv_fp8_e4m3 x;
      x.__x = static_cast<__nv_fp8_storage_t>(w >> (8 * (i % 4)));
      f[i] = static_cast<float>(x);
    }
  }
}

__global__ void __launch_bounds__(256) chunk_attn_kernel(ChunkAttnArgs a) {
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  const int row = blockIdx.x, lane = threadIdx.x & 31;
  const int head = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (row == 0 && head < 8) {
    for (int b = threadIdx.x; b < a.batch; b += 256) {
      const int s0 = a.q_start[b], s1 = a.q_start[b + 1];
      if (s0 < 0 || s1 < s0 || s1 > a.n_rows) atomicOr(a.err, kErrLayout);
    }
  }
  int seq = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 256)
    seq += __syncthreads_count(b0 + threadIdx.x < a.batch &&
                               a.q_start[b0 + threadIdx.x + 1] <= row);
  if (seq >= a.batch || row < a.q_start[seq]) return;
  const KvSeq& s = a.kv[seq];
  if (s.page_size != a.page_size || s.chunk_maps == 0) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrLayout);
    return;
  }
  const int n = a.q_start[seq + 1] - a.q_start[seq], L = a.seq_lens[seq];
  const size_t o_at = (static_cast<size_t>(row) * kHeads + head) * kHeadDim + 8 * lane;
  const uint32_t bits = a.q_start[seq + 1] > a.n_rows || a.q_start[seq] < 0 ? kErrLayout
                        : L > s.capacity              ? kErrCapacity
                        : L < n                       ? kErrEmpty
                                                      : 0u;
  if (bits != 0) {
    if (threadIdx.x == 0) atomicOr(a.err, bits);
    *reinterpret_cast<uint4*>(a.out + o_at) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int last = L - (a.q_start[seq + 1] - row);
  float q[8], o[8], m = -INFINITY, l = 0.f;
  {
    KvSeq none{};
    load8(none, a.q, MFA_KV_BF16, static_cast<long long>(row) * kHeads + head, lane, q);
  }
  const bool fp8 = a.kv_dtype == MFA_KV_FP8_E4M3;
  const float mul = a.scale * kLog2e * (fp8 ? a.k_scale : 1.f);
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  for (int j = 0; j <= last; ++j) {
    const long long at = kv_row_index(s, j);
    float k[8] = {}, v[8] = {};
    if (at >= 0) {
      load8(s, s.k, a.kv_dtype, at, lane, k);
      load8(s, s.v, a.kv_dtype, at, lane, v);
    }
    float x = 0.f;
    for (int i = 0; i < 8; ++i) x = fmaf(q[i], k[i], x);
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= mul;
    const float mn = fmaxf(m, x), base = mn == -INFINITY ? 0.f : mn;
    const float w = exp2f(x - base), al = exp2f(m - base);
    l = fmaf(l, al, w);
    for (int i = 0; i < 8; ++i) o[i] = fmaf(o[i], al, w * v[i]);
    m = mn;
  }
  const float r = (fp8 ? a.v_scale : 1.f) / l;
  uint32_t w[4];
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i] * r, o[2 * i + 1] * r);
    w[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(a.out + o_at) = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace

cudaError_t launch_chunk_attn(const ChunkAttnArgs& a, cudaStream_t s) {
  return launch_pdl(chunk_attn_kernel, dim3(a.n_rows, kHeads / 8), dim3(256), 0, s, a);
}

}  // namespace mfa
