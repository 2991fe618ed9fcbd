// Attention of one new token per sequence over the paged e4m3 cache: one warp
// per (sequence, head), online softmax.
#include "common.cuh"

namespace cslc {

__global__ void __launch_bounds__(256) page_decode_kernel(
    const uint16_t* __restrict__ q, const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
    const float* __restrict__ k_scale, const float* __restrict__ v_scale, const int32_t* __restrict__ table,
    const int32_t* __restrict__ seq_len, int B, int H, int Hkv, int P, int n_pages, int max_pages, long long q_stride,
    int window, float scale, uint16_t* __restrict__ out, float* __restrict__ lse) {
  const int row = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (row >= B * H) return;
  const int b = row / H, h = row % H, hk = h / (H / Hkv);
  const long long cap = (long long)max_pages * P;
  const int n = (int)min((long long)max(seq_len[b], 0), cap);
  const int lo = window > 0 ? max(0, n - window) : 0;
  const uint2 qv = reinterpret_cast<const uint2*>(q + b * q_stride + (long long)h * kD)[lane];
  const float qf[4] = {bf16_lo(qv.x), bf16_hi(qv.x), bf16_lo(qv.y), bf16_hi(qv.y)};
  auto decode = [](uint32_t u, float s, float (&f)[4]) {
    const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u & 0xffffu), __NV_E4M3)));
    const float2 c = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> 16), __NV_E4M3)));
    f[0] = a.x * s; f[1] = a.y * s; f[2] = c.x * s; f[3] = c.y * s;
  };
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = lo; j < n; ++j) {
    const int p = table[(size_t)b * max_pages + j / P];
    if (p < 0 || p >= n_pages) continue;
    const size_t ps = (size_t)p * Hkv + hk, at = (ps * P + j % P) * kD;
    float kf[4], vf[4];
    decode(reinterpret_cast<const uint32_t*>(k_cache + at)[lane], k_scale[ps], kf);
    decode(reinterpret_cast<const uint32_t*>(v_cache + at)[lane], v_scale[ps], vf);
    const float s = warp_sum(qf[0] * kf[0] + qf[1] * kf[1] + qf[2] * kf[2] + qf[3] * kf[3]) * scale;
    const float mn = fmaxf(m, s);
    const float a = mn == -INFINITY ? 1.f : expf(m - mn), e = mn == -INFINITY ? 0.f : expf(s - mn);
    m = mn;
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(e, vf[i], o[i] * a);
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  reinterpret_cast<uint2*>(out + (size_t)row * kD)[lane] =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (lse != nullptr && lane == 0) lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

size_t page_decode_workspace_bytes(int, int, int) { return 0; }

cslc_status launch_page_decode(const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                               const float* v_scale, const int32_t* table, const int32_t* seq_len, int B, int H,
                               int Hkv, int page, int n_pages, int max_pages, long long q_stride, int window,
                               float scale, uint16_t* out, float* lse, void*, cudaStream_t stream) {
  page_decode_kernel<<<(B * H + 7) / 8, 256, 0, stream>>>(q, k_cache, v_cache, k_scale, v_scale, table, seq_len, B, H,
                                                          Hkv, page, n_pages, max_pages, q_stride, window, scale, out,
                                                          lse);
  return check_launch("page_decode_kernel");
}

}  // namespace cslc
