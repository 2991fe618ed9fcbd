// The page plan and the cache write of the paged e4m3 cache.
//
// Plan: sequence b grows from old[b] to old[b] + new[b] tokens. Its pages
// p0 = ceil(old / P) .. p1 - 1 (p1 = ceil((old + new) / P), at most max_pages)
// come from the free list in sequence order, so page p0 + i of sequence b is
// free[ex_b + i] with ex the exclusive scan of p1 - p0; token x of the sequence
// gets slot table[b, x / P] * P + x mod P. Every CTA scans all lengths itself
// (B <= 8192: at most 64 KB from L2) instead of waiting for another CTA, so
// the plan is one launch without a workspace; it is bound by latency: 3.5 us in a
// captured graph for 64 requests of one token, 5.8 us for 512 with 54,211 tokens (a
// call of its own takes the host 8.7 us).
//
// Write: a run is a stretch of consecutive tokens with consecutive slots of
// one page; it is the unit of work, for each head and each of K and V. The
// scale of a page is a power of two 2^e: e the smallest exponent with
// amax <= 448 * 2^e. A power of two costs no precision (the codes are floating
// point, only their range shifts), makes code * scale exact in bf16, and lets
// a page whose later tokens are larger move its earlier codes to the new
// scale without a second rounding (but for those that become subnormal).
// One CTA holds a run in registers between the maximum and the conversion, so
// the input is read once; HBM bound: 65,536 tokens of 8 heads 68.1-69.6 us (5.8-5.9
// TB/s, 90-91 % of a copy's rate), 13 prompts of up to 2,001 tokens 20.8 us (16.3 us in
// a captured graph, 92 %).

#include "dependent.cuh"

namespace cslc {

namespace {

constexpr int PP_THREADS = 512;
constexpr int PP_TOKENS = 512;         // slots of one CTA: one to a thread
constexpr int PP_MAX_B = 8192;

// Inclusive scan of (a, b) over the block, saturating sums kept in 64 bits.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long (*wsum)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) { a += x; b += y; }
  }
  if (lane == 31) { wsum[warp][0] = a; wsum[warp][1] = b; }
  __syncthreads();
  for (int w = 0; w < warp; ++w) { a += wsum[w][0]; b += wsum[w][1]; }
  __syncthreads();
}

__device__ __forceinline__ int sat32(long long x) { return x > 0x7fffffffll ? 0x7fffffff : (int)x; }

}  // namespace

__global__ void __launch_bounds__(PP_THREADS) page_plan_kernel(
    const int32_t* __restrict__ old_len, const int32_t* __restrict__ new_len, int B,
    const int32_t* __restrict__ free_pages, int n_free, int page_log2, int n_pages, int max_pages, int max_tokens,
    int32_t* __restrict__ table, int32_t* __restrict__ slots, int32_t* __restrict__ cu,
    int32_t* __restrict__ seq_len, int32_t* __restrict__ status) {
  extern __shared__ int32_t pp_smem[];
  grid_dependency_wait();
  int32_t* tok = pp_smem;              // [B + 1] tokens before sequence b
  int32_t* pg = tok + B + 1;           // [B + 1] pages handed out before sequence b
  __shared__ long long wsum[PP_THREADS / 32][2];
  __shared__ unsigned long long lost_s;   // lengths of any int32 value: more than 32 bits hold
  const int tid = threadIdx.x;
  const int P = 1 << page_log2;
  const int per = (B + PP_THREADS - 1) / PP_THREADS;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  auto first_page = [&](int b) { return (int)(((long long)max(old_len[b], 0) + P - 1) >> page_log2); };
  auto end_page = [&](int b) {
    const long long n = (long long)max(old_len[b], 0) + max(new_len[b], 0);
    return (int)min((long long)max_pages, (n + P - 1) >> page_log2);
  };
  long long st = 0, sp = 0;
  for (int b = b0; b < b1; ++b) { st += max(new_len[b], 0); sp += max(0, end_page(b) - first_page(b)); }
  long long it = st, ip = sp;
  if (tid == 0) lost_s = 0;
  block_scan2(it, ip, wsum);
  it -= st;
  ip -= sp;
  for (int b = b0; b < b1; ++b) {
    tok[b] = sat32(it);
    pg[b] = sat32(ip);
    it += max(new_len[b], 0);
    ip += max(0, end_page(b) - first_page(b));
  }
  if (b0 < B && b1 == B) { tok[B] = sat32(it); pg[B] = sat32(ip); }
  if (B == 0 && tid == 0) { tok[0] = 0; pg[0] = 0; }
  __syncthreads();
  const int T = tok[B], taken = pg[B];
  auto given = [&](long long i) {       // page i of those handed out, -1 where there is none
    if (i >= n_free) return -1;
    const int p = free_pages[i];
    return p >= 0 && p < n_pages ? p : -1;
  };
  auto owner = [&](const int32_t* before, int x) {   // the last b with before[b] <= x
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
  };
  const long long step = gridDim.x * PP_THREADS, at = blockIdx.x * PP_THREADS + tid;   // the sizes go up to 2^31 - 1
  // new entries of the tables
  for (long long i = at; i < taken; i += step) {
    const int b = owner(pg, (int)i);
    table[(size_t)b * max_pages + first_page(b) + (i - pg[b])] = given(i);
  }
  // slots; entries below p0 are the caller's and no CTA writes them
  for (long long t = at; t < max_tokens; t += step) {
    int slot = -1;
    if (t < T) {
      const int b = owner(tok, (int)t);
      const long long x = (long long)max(old_len[b], 0) + (t - tok[b]);
      const long long j = x >> page_log2;
      if (j < max_pages) {
        const int p0 = first_page(b);
        int p = j < p0 ? table[(size_t)b * max_pages + j] : given((long long)pg[b] + (j - p0));
        if (p >= 0 && p < n_pages) slot = p * P + (int)(x & (P - 1));
      }
    }
    slots[t] = slot;
  }
  if (blockIdx.x != 0) return;
  long long lost = 0;
  for (int b = tid; b < B; b += PP_THREADS) {
    cu[b] = tok[b];
    const long long o = max(old_len[b], 0), n = max(new_len[b], 0);
    seq_len[b] = sat32(o + n);
    // tokens before the first page that is missing: a missing partial page loses its own tokens only
    const int p0 = first_page(b), p1 = end_page(b);
    const int have = max(0, min(p1 - p0, n_free - min(pg[b], n_free)));
    long long covered = max(0ll, min(o + n, (long long)(p0 + have) << page_log2) - o);
    if ((o >> page_log2) >= max_pages) {
      covered = 0;
    } else if ((o & (P - 1)) != 0 && n > 0) {
      const int p = table[(size_t)b * max_pages + (o >> page_log2)];
      if (p < 0 || p >= n_pages) covered -= min(n, ((long long)p0 << page_log2) - o);
    }
    lost += n - covered;
  }
  // pages of the free list that are no pages
  for (long long i = tid; i < min(taken, n_free); i += PP_THREADS)
    if (given(i) < 0) {
      const int b = owner(pg, (int)i);
      const long long x0 = ((long long)first_page(b) + (i - pg[b])) << page_log2;
      const long long o = max(old_len[b], 0), end = o + max(new_len[b], 0);
      lost += min(end, x0 + P) - x0;
    }
  if (lost) atomicAdd(&lost_s, (unsigned long long)lost);
  __syncthreads();
  if (tid == 0) {
    cu[B] = T;
    status[0] = taken;
    status[1] = sat32((long long)lost_s);
  }
}

cslc_status launch_page_plan(const int32_t* old_len, const int32_t* new_len, int B, const int32_t* free_pages,
                             int n_free, int page, int n_pages, int max_pages, int max_tokens, int32_t* table,
                             int32_t* slots, int32_t* cu, int32_t* seq_len, int32_t* status, cudaStream_t stream) {
  const size_t smem = (size_t)(B + 1) * 2 * sizeof(int32_t);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return set_error(CSLC_ERR_CUDA, "cslc_page_plan: %s", cudaGetErrorString(e));
  }
  const int want = max_tokens / PP_TOKENS + 1;
  const int grid = want > 148 ? 148 : want;
  const cudaError_t e = launch_after(page_plan_kernel, dim3(grid), dim3(PP_THREADS), smem, stream, old_len, new_len, B,
                                         free_pages, n_free, 31 - __builtin_clz(page), n_pages, max_pages, max_tokens,
                                         table, slots, cu, seq_len, status);
  if (e != cudaSuccess) return set_error(CSLC_ERR_CUDA, "page_plan_kernel: %s", cudaGetErrorString(e));
  return CSLC_OK;
}

// ---------------------------------------------------------------- cache write

namespace {

constexpr int PW_THREADS = 256;             // at most: 2 P threads, 4 pieces of 16 dims each, hold a page
constexpr int PW_MAX_PAGE = 128;

// The smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8), held to the range.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kScaleExpMin), kScaleExpMax);
}
// The larger absolute values of two pairs of bf16 (a NaN loses), and the same without
// infinities: a magnitude of 0x7f80 and more is no number.
__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t x) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
  return r;
}
__device__ __forceinline__ uint32_t only_finite2(uint32_t x) {
  const uint32_t a = x & 0x7fff7fffu;
  return ((a & 0xffffu) < 0x7f80u ? a & 0xffffu : 0u) | (a < 0x7f800000u ? a & 0xffff0000u : 0u);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ float4 from_e4m3x4(uint32_t v) {
  const __half2 lo = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v & 0xffffu), __NV_E4M3));
  const __half2 hi = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v >> 16), __NV_E4M3));
  const float2 a = __half22float2(lo), b = __half22float2(hi);
  return make_float4(a.x, a.y, b.x, b.y);
}

}  // namespace

// Grid: windows of W tokens x (K and V of the heads), the latter fastest so that
// neighbouring CTAs read neighbouring memory. A CTA takes the runs that begin in its window.
__global__ void __launch_bounds__(PW_THREADS, 4) page_write_kernel(
    const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, const int32_t* __restrict__ slots, int T, int W,
    int R, int Hkv, int page_log2, int n_pages, long long k_stride, long long v_stride, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, float* __restrict__ k_scale, float* __restrict__ v_scale) {
  grid_dependency_wait();
  __shared__ int s_slot[2 * PW_MAX_PAGE + 1];            // slots of tokens w0 - 1 .. w0 + W + P - 1
  __shared__ uint32_t s_break[2 * PW_MAX_PAGE / 32 + 1]; // bit t: token w0 + t does not continue a run
  __shared__ float s_max[PW_THREADS / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
  const int P = 1 << page_log2;
  const int groups = 2 * Hkv / R;                        // of R heads of K or V each
  const int y0 = blockIdx.x % groups * R, w0 = blockIdx.x / groups * W;

  const int n = W + P;                                   // at most 2 P
  for (int i = tid; i < n + 1; i += threads) {
    const int t = w0 - 1 + i;
    int s = t >= 0 && t < T ? slots[t] : -1;
    if (s >= 0 && (s >> page_log2) >= n_pages) s = -1;
    s_slot[i] = s;
  }
  __syncthreads();
  {
    const int i = tid;                                   // token w0 + i
    bool brk = true;
    if (i < n) {
      const int s = s_slot[i + 1];
      brk = s < 0 || s_slot[i] < 0 || s != s_slot[i] + 1 || (s & (P - 1)) == 0;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, brk);
    if (lane == 0) s_break[warp] = m;
    if (tid == 0) s_break[threads / 32] = 0xffffffffu;
  }
  __syncthreads();

  auto next_break = [&](int t) {                         // the first one at or behind t (one is behind the last token)
    int wd = t >> 5;
    uint32_t m = s_break[wd] & (0xffffffffu << (t & 31));
    while (m == 0u) m = s_break[++wd];
    return wd * 32 + __ffs(m) - 1;
  };
  for (int i = next_break(0), end; i < W; i = end) {     // uniform over the CTA
    end = next_break(i + 1);
    const int slot = s_slot[i + 1];
    if (slot < 0) continue;
    const int len = end - i;                             // <= P: a run ends at its page's end
    const int pid = slot >> page_log2, o = slot & (P - 1);
    for (int y = y0; y < y0 + R; ++y) {
      const bool is_v = y >= Hkv;
      const int head = is_v ? y - Hkv : y;
      const uint16_t* src = (is_v ? v : k) + head * kD;
      const long long stride = is_v ? v_stride : k_stride;
      uint8_t* cache = is_v ? v_cache : k_cache;
      float* scale = is_v ? v_scale : k_scale;
      const size_t ps = (size_t)pid * Hkv + head;
      uint8_t* dst = cache + (ps << page_log2) * kD;
      const uint16_t* run = src + (long long)(w0 + i) * stride;

      const float old_scale = o > 0 ? scale[ps] : 0.f;
      uint4 x[4][2];                                       // up to 4 pieces of 16 dims
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tid + j * threads;                 // row c / 8, dims 16 (c mod 8) ..
        if (c < len * 8) {
          const uint4* p = reinterpret_cast<const uint4*>(run + (long long)(c >> 3) * stride + (c & 7) * 16);
          x[j][0] = __ldcs(p);
          x[j][1] = __ldcs(p + 1);
        } else {
          x[j][0] = x[j][1] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      uint32_t m2 = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          m2 = absmax2(absmax2(absmax2(absmax2(m2, x[j][h].x), x[j][h].y), x[j][h].z), x[j][h].w);
      if (__any_sync(0xffffffffu, (m2 & 0xffffu) == 0x7f80u || (m2 >> 16) == 0x7f80u)) {   // an infinity: leave it out
        m2 = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            m2 = absmax2(absmax2(m2, only_finite2(x[j][h].x)), only_finite2(x[j][h].y));
            m2 = absmax2(absmax2(m2, only_finite2(x[j][h].z)), only_finite2(x[j][h].w));
          }
      }
      float amax = fmaxf(bf16_lo(m2), bf16_hi(m2));
      amax = warp_max(amax);
      if (lane == 0) s_max[warp] = amax;
      __syncthreads();
      for (int w = 0; w < threads / 32; ++w) amax = fmaxf(amax, s_max[w]);
      int e = scale_exponent(amax);
      if (o > 0) {
        const int e_old = page_scale_exponent(old_scale);
        e = max(e, e_old);
        if (e > e_old) {
          const float f = pow2(max(e_old - e, -120));
          for (int c = tid; c < o * 8; c += threads) {
            uint4* p = reinterpret_cast<uint4*>(dst + (size_t)c * 16);
            uint4 u = *p;
            uint32_t* w4 = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 g = from_e4m3x4(w4[q]);
              w4[q] = e4m3x4(g.x * f, g.y * f, g.z * f, g.w * f);
            }
            *p = u;
          }
        }
      }
      const float inv = pow2(-e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tid + j * threads;
        if (c < len * 8) {
          uint4 u;
          uint32_t* w4 = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t in[4] = {x[j][h].x, x[j][h].y, x[j][h].z, x[j][h].w};
#pragma unroll
            for (int q = 0; q < 2; ++q)
              w4[2 * h + q] = e4m3x4(bf16_lo(in[2 * q]) * inv, bf16_hi(in[2 * q]) * inv, bf16_lo(in[2 * q + 1]) * inv,
                                     bf16_hi(in[2 * q + 1]) * inv);
          }
          *reinterpret_cast<uint4*>(dst + (size_t)o * kD + (size_t)c * 16) = u;
        }
      }
      __syncthreads();                                     // every thread has read the old scale and s_max
      if (tid == 0) scale[ps] = pow2(e);
    }
  }
}

cslc_status launch_page_write(const uint16_t* k, const uint16_t* v, const int32_t* slots, int T, int Hkv, int page,
                              int n_pages, long long k_stride, long long v_stride, uint8_t* k_cache, uint8_t* v_cache,
                              float* k_scale, float* v_scale, cudaStream_t stream) {
  // A window of a page where that fills the GPU, of fewer tokens where it does not (a step of
  // 64 single tokens would be one block's).
  int W = page;
  while (W > 1 && (long long)((T + W - 1) / W) * 2 * Hkv < 4 * 148) W >>= 1;
  // Several heads to a CTA, which then reads the slots once, while CTAs for every SM remain:
  // pages of 128, 65,536 tokens of 8 heads: 1 / 2 / 4 / 8 heads 82.8 / 75.7 / 73.5 / 70.1 us. The smaller
  // CTAs of smaller pages want more of them beyond two heads: pages of 64, 40,000 tokens of
  // 16 heads: 2 / 4 / 8 heads 81.0 / 80.6 / 89.9 us, and 15,845 tokens of 8: 1 / 2 / 4 heads 22.5 / 21.4 / 26.7.
  const int threads = page < 32 ? 64 : 2 * page, once = 148 * (1024 / threads);   // CTAs that run at a time
  int R = 1;
  while (R < 8 && (2 * Hkv) % (2 * R) == 0 &&
         (long long)((T + W - 1) / W) * (2 * Hkv / (2 * R)) >= (page == PW_MAX_PAGE || R == 1 ? once : once * 5 / 2))
    R *= 2;
  const unsigned grid = (unsigned)((T + W - 1) / W) * (unsigned)(2 * Hkv / R);
  const cudaError_t e = launch_after(page_write_kernel, dim3(grid), dim3(threads), 0, stream, k, v,
                                         slots, T, W, R, Hkv, 31 - __builtin_clz(page), n_pages, k_stride, v_stride,
                                         k_cache, v_cache, k_scale, v_scale);
  if (e != cudaSuccess) return set_error(CSLC_ERR_CUDA, "page_write_kernel: %s", cudaGetErrorString(e));
  return CSLC_OK;
}

}  // namespace cslc
