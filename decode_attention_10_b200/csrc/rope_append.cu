// Rotation of a chunk of new tokens' queries and keys, and the append of their keys and
// values to the KV cache, in one pass over the data (include/mfa.h: mfa_rope_append).
//
// Pair i of a row, (a, b), becomes (a cos - b sin, b cos + a sin) with the cosine and sine of
// position p of the token on the pair's axis, read from the caller's table: angles of far
// positions need more than float32 to form, so the table is made once, in float64, and the
// kernel only multiplies (float32, one rounding at the end).
//
// One block per token. A row of 256 dimensions is 16 units of 16 dimensions -- a unit is
// eight whole pairs, so a thread rotates what it has loaded. Thread (group, unit) takes its
// unit of 64 / groups heads, all its 16-byte loads in flight before anything is waited for.
// Groups 0 and 1 take the K and the V row as well. Everything a token needs to know (its
// sequence, cache row, page and angles) is looked up while its 32 KB of queries arrive; the
// angles are shared by the block through shared memory, since all 65 rows turn by the same
// ones.
//
// Bound by HBM: 32 KB in and out a token. Blocks of 128 threads (8 heads and sixteen 16-byte
// loads a thread, 4 blocks an SM) move 6.5 TB/s, all of a copy's rate: 8409 tokens, bf16 cache,
// 88.8 us; 256 threads (4 heads) 113 us, 512 (2 heads) 168 us, since a block's chain of
// look-ups is then paid for fewer bytes a thread. Where the tokens fill no more than the SMs,
// that chain is all there is, and more threads a block shorten it (kSmallRows).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "chunk.cuh"
#include "sm100.cuh"

namespace mfa {
namespace {

constexpr int kUnits = kHeadDim / 16;  // 16-dimension units of a row
constexpr int kMaxPairs = kHeadDim / 2;
// Up to one token an SM, blocks of 512 threads; above it blocks of 128. Measured at 64, 148,
// 200 and 444 tokens: 3.3, 3.3, 5.7, 10.1 us with 512 threads, 3.9, 5.0, 5.2, 6.8 with 128.
constexpr int kSmallRows = 148;

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

struct Row16 {  // the 16 dimensions of a unit, in float32: its first and second eight
  float a[8], b[8];
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Rotate a unit's eight pairs: (a[i], b[i]), or for neighbouring pairs (a[2i], a[2i+1]) and
// (b[2i], b[2i+1]).
__device__ __forceinline__ void rotate(Row16& r, const float (&c)[8], const float (&s)[8],
                                       bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = r.a[2 * i], y0 = r.a[2 * i + 1];
      r.a[2 * i] = x0 * c[i] - y0 * s[i];
      r.a[2 * i + 1] = y0 * c[i] + x0 * s[i];
      const float x1 = r.b[2 * i], y1 = r.b[2 * i + 1];
      r.b[2 * i] = x1 * c[i + 4] - y1 * s[i + 4];
      r.b[2 * i + 1] = y1 * c[i + 4] + x1 * s[i + 4];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = r.a[i], y = r.b[i];
      r.a[i] = x * c[i] - y * s[i];
      r.b[i] = y * c[i] + x * s[i];
    }
  }
}

// Eight values as e4m3(value / scale), the append's rounding (one float32 division, one
// rounding to nearest even, saturating).
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8], float scale) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i / 4] |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(__fdiv_rn(f[i], scale),
                                                            __NV_SATFINITE, __NV_E4M3))
                << (8 * (i % 4));
  return make_uint2(w[0], w[1]);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads)
    rope_append_kernel(const __grid_constant__ RopeAppendArgs a) {
  constexpr int kGroups = kThreads / kUnits;     // groups of heads
  constexpr int kGroupHeads = kHeads / kGroups;  // heads of a thread
  static_assert(kGroups >= 2 && kThreads >= kMaxPairs, "K, V and the angles each in one go");
  __shared__ __align__(16) float s_cos[kMaxPairs], s_sin[kMaxPairs];
  const int row = blockIdx.x, tid = threadIdx.x;
  const int u = tid % kUnits, group = tid / kUnits;
  const int pairs = a.rot_dim / 2;
  // this unit's two runs of eight dimensions, and whether it is rotated
  const bool turn = 16 * u < a.rot_dim;
  const bool split = turn && !a.interleaved;
  const int d0 = split ? 8 * u : 16 * u;
  const int d1 = split ? pairs + 8 * u : 16 * u + 8;

  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  // the data first: it depends on nothing but the row
  uint4 q0[kGroupHeads], q1[kGroupHeads], x0, x1;
  const size_t q_at = (static_cast<size_t>(row) * kHeads + group * kGroupHeads) * kHeadDim;
  if (a.q != nullptr) {
#pragma unroll
    for (int h = 0; h < kGroupHeads; ++h) {
      q0[h] = *reinterpret_cast<const uint4*>(a.q + q_at + h * kHeadDim + d0);
      q1[h] = *reinterpret_cast<const uint4*>(a.q + q_at + h * kHeadDim + d1);
    }
  }
  // groups 0 and 1: the token's K and V rows (V in plain runs of 16)
  if (group < 2) {
    const uint16_t* src = group == 0 ? a.k + static_cast<size_t>(row) * a.k_ld
                                     : a.v + static_cast<size_t>(row) * a.v_ld;
    x0 = *reinterpret_cast<const uint4*>(src + (group == 0 ? d0 : 16 * u));
    x1 = *reinterpret_cast<const uint4*>(src + (group == 0 ? d1 : 16 * u + 8));
  }
  int pos = 0;  // of this thread's pair (tid < pairs)
  if (a.positions != nullptr && tid < pairs)
    pos = a.positions[static_cast<size_t>(a.pair_axis[tid]) * a.n_rows + row];
  // the token's sequence: as many as end at or before this row (one round trip; sequences
  // without new tokens end where they begin and are passed over). Every block looks all ranges of
  // rows over: where they do not hold together, none writes.
  int seq = 0;
  bool layout = false;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    bool ends = false;
    if (b0 + tid < a.batch) {
      const int s0 = a.q_start[b0 + tid], s1 = a.q_start[b0 + tid + 1];
      layout |= s0 < 0 || s1 < s0 || s1 > a.n_rows;
      ends = s1 <= row;
    }
    seq += __syncthreads_count(ends);
  }
  if (layout && row == 0) atomicOr(a.err, kErrLayout);
  if (seq >= a.batch || row < a.q_start[seq]) return;  // the row belongs to no sequence
  const KvSeq* kv = a.kv + seq;
  const int place = a.seq_lens[seq] - (a.q_start[seq + 1] - row);  // the cache row
  const long long at = kv_row_index(*kv, place);
  if (a.positions == nullptr) pos = place;
  const bool bad_pos = tid < pairs && (pos < 0 || pos >= a.max_pos);
  if (tid < pairs && !bad_pos) {
    const float* t = a.table + static_cast<size_t>(pos) * a.rot_dim;
    s_cos[tid] = t[tid];
    s_sin[tid] = t[pairs + tid];
  }
  // (also the barrier before the angles are read)
  if (__syncthreads_or(bad_pos || at < 0 || layout)) {
    const bool refused = __syncthreads_or(layout);
    if (tid == 0 && !refused) atomicOr(a.err, kErrCapacity);
    return;
  }
  float c[8], s[8];
  if (turn) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 cv = *reinterpret_cast<const float4*>(s_cos + 8 * u + 4 * i);
      const float4 sv = *reinterpret_cast<const float4*>(s_sin + 8 * u + 4 * i);
      c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
      s[4 * i] = sv.x, s[4 * i + 1] = sv.y, s[4 * i + 2] = sv.z, s[4 * i + 3] = sv.w;
    }
  }
  if (group < 2) {
    const bool is_k = group == 0;
    const int e0 = is_k ? d0 : 16 * u, e1 = is_k ? d1 : 16 * u + 8;
    Row16 r;
    unpack8(x0, r.a);
    unpack8(x1, r.b);
    if (is_k && turn) rotate(r, c, s, a.interleaved);
    if (a.kv_dtype == MFA_KV_BF16) {
      uint16_t* dst = static_cast<uint16_t*>(is_k ? kv->k : kv->v) + at * kHeadDim;
      *reinterpret_cast<uint4*>(dst + e0) = pack8(r.a);
      *reinterpret_cast<uint4*>(dst + e1) = pack8(r.b);
    } else {
      uint8_t* dst = static_cast<uint8_t*>(is_k ? kv->k : kv->v) + at * kHeadDim;
      const float scale = is_k ? a.k_scale : a.v_scale;
      *reinterpret_cast<uint2*>(dst + e0) = pack8_e4m3(r.a, scale);
      *reinterpret_cast<uint2*>(dst + e1) = pack8_e4m3(r.b, scale);
    }
  }
  if (a.q == nullptr || (!turn && a.q_out == a.q)) return;
#pragma unroll
  for (int h = 0; h < kGroupHeads; ++h) {
    if (turn) {
      Row16 r;
      unpack8(q0[h], r.a);
      unpack8(q1[h], r.b);
      rotate(r, c, s, a.interleaved);
      q0[h] = pack8(r.a);
      q1[h] = pack8(r.b);
    }
    *reinterpret_cast<uint4*>(a.q_out + q_at + h * kHeadDim + d0) = q0[h];
    *reinterpret_cast<uint4*>(a.q_out + q_at + h * kHeadDim + d1) = q1[h];
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t s) {
  if (a.n_rows <= kSmallRows)
    return launch_pdl(rope_append_kernel<512>, dim3(a.n_rows), dim3(512), 0, s, a);
  return launch_pdl(rope_append_kernel<128>, dim3(a.n_rows), dim3(128), 0, s, a);
}

}  // namespace mfa
