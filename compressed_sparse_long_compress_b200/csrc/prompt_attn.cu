// Causal attention of packed sequences: one warp per query row, online softmax.
#include "common.cuh"

namespace cslc {

__global__ void __launch_bounds__(256) prompt_attn_kernel(
    const uint16_t* __restrict__ q, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
    const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, int B, int Tq, int Tk, int H, int Hkv,
    long long q_stride, long long k_stride, long long v_stride, int window, float scale, uint16_t* __restrict__ out,
    float* __restrict__ lse) {
  const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= (long long)Tq * H) return;
  const int t = (int)(row / H), h = (int)(row % H), hk = h / (H / Hkv);
  int b = 0;
  while (b < B && !(t >= cu_q[b] && t < cu_q[b + 1])) ++b;
  if (b == B) return;
  const int nq = cu_q[b + 1] - cu_q[b];
  const int k0 = min(max(cu_k[b], 0), Tk), k1 = min(max(cu_k[b + 1], k0), Tk);
  const int nk = k1 - k0;
  const int last = t - cu_q[b] + nk - nq;
  const int lo = window > 0 ? max(0, last - window + 1) : 0;
  const uint2 qv = reinterpret_cast<const uint2*>(q + t * q_stride + (long long)h * kD)[lane];
  const float qf[4] = {bf16_lo(qv.x), bf16_hi(qv.x), bf16_lo(qv.y), bf16_hi(qv.y)};
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = lo; j <= last; ++j) {
    const uint2 kv = reinterpret_cast<const uint2*>(k + (k0 + j) * k_stride + (long long)hk * kD)[lane];
    const uint2 vv = reinterpret_cast<const uint2*>(v + (k0 + j) * v_stride + (long long)hk * kD)[lane];
    const float s = warp_sum(qf[0] * bf16_lo(kv.x) + qf[1] * bf16_hi(kv.x) + qf[2] * bf16_lo(kv.y) +
                             qf[3] * bf16_hi(kv.y)) * scale;
    const float mn = fmaxf(m, s);
    const float a = mn == -INFINITY ? 1.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
    m = mn;
    l = l * a + p;
    const float vf[4] = {bf16_lo(vv.x), bf16_hi(vv.x), bf16_lo(vv.y), bf16_hi(vv.y)};
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(p, vf[i], o[i] * a);
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  reinterpret_cast<uint2*>(out + row * kD)[lane] =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (lse != nullptr && lane == 0) lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

size_t prompt_attn_workspace_bytes(int, int, int, int) { return 0; }

cslc_status launch_prompt_attn(const uint16_t* q, const uint16_t* k, const uint16_t* v, const int32_t* cu_q,
                               const int32_t* cu_k, int B, int Tq, int Tk, int H, int Hkv, long long q_stride,
                               long long k_stride, long long v_stride, int window, float scale, uint16_t* out,
                               float* lse, void*, cudaStream_t stream) {
  const long long rows = (long long)Tq * H;
  prompt_attn_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(q, k, v, cu_q, cu_k, B, Tq, Tk, H, Hkv, q_stride,
                                                                     k_stride, v_stride, window, scale, out, lse);
  return check_launch("prompt_attn_kernel");
}

}  // namespace cslc
