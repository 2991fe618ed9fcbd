// Attention of one new token per sequence over the paged e4m3 cache, on the
// 5th-generation tensor cores (tcgen05 + TMEM).
//
// Mathematics. A tile is 128 consecutive tokens of a sequence; a unit is one
// (sequence, key head, group of up to GP query heads). The codes are operands
// as they lie in the cache, without a conversion:
//   S^T[token, head] = K[token, dim] q[head, dim]       (M = 128 tokens)
//   O^T[dim, head]   = V^T[dim, token] P[token, head]   (M = 128 dims; V MN-major)
// q and P have 8 significant bits and e4m3 has 4, so each is split into two
// e4m3 parts that sit side by side as N = 2 GP columns: x = hi + lo / 16, hi =
// e4m3(x), lo = e4m3(16 (x - hi)). From 2^-6 on that is what a rounding to 8
// significant bits would be (2^-8 of x, exact for a bf16); below, hi is subnormal
// and x off by at most 2^-14. q is scaled by a power of two to [128, 256) at
// its row's largest: components from 2^-13 of that one on are exact, smaller ones off
// by at most 2^-21 of it (a row whose largest is below 2^-110 is scaled less and has
// fewer bits). Page scales are powers of two: k's multiplies the score, v's
// is added to the score's exponent before the exponential, so P V needs no
// scale of its own, and is taken out again (times 2^-e) for the softmax sum. Score
// and exponent are rounded to fp32 as one number: half a step of the score, so that
// from about 2^16 on equal scores in pages of different V scales weigh apart by that.
// Each tile has its own reference (its exact maximum, mapped to 2^7 .. 2^8): the O^T
// of a tile is a fresh product, rescaled as it joins the fp32 sum in registers.
// So a probability is off by at most 2^-8 of itself and 2^-21 of the largest one of
// its own tile, however flat and long the tail is; a running reference would lose
// tails of 2^-23 per token.
//
// Work. All tiles of all units, in the order of the sequences, are dealt to the
// CTAs in equal consecutive ranges (two or three CTAs per SM), whatever the lengths are;
// a unit counts PD_UNIT tiles more for its start and end.
// A unit that crosses CTAs leaves fp32 partials in the workspace, which
// page_decode_combine_kernel (a programmatic dependent launch) merges. Short units
// (small windows, short tables) of one turn of CTAs go to a CTA each, without that.
//
// Measured (64 heads on 8, pages of 128 and 64): 8 requests of up to 131,072 tokens
// 217-221 us (6.1-6.2 TB/s of codes and scales, 95-97 % of a copy's rate), 64 of up to
// 8,192 tokens 95-98 us (83-85 %): bound by HBM while the CTAs run; the rest is their
// start, the units' ends and the merge. 16 heads to a key head are bound by the softmax's
// instructions: 64 requests of up to 8,192 tokens, 128 heads on 8, 117-121 us where the
// bytes take 82. Larger groups read the cache once for each 16 heads, every time so
// bound: 64 heads on one key head 66 us where the bytes take 10.4, 128 on one 113.
//
// CTA roles: warps 0-3 softmax (thread = token, then = dim), warp 4 producer
// (page table and scales, one tile ahead; TMA of each page's codes, STAGES-deep
// ring; the parts of q, a segment ahead), warp 5 TMEM allocation and the
// MMA-issuing thread. Tokens outside
// the sequence's visible range get P = 0 and their V rows are cleared in shared memory,
// since stale codes may be NaN. All waits are time-bounded.

#include "dependent.cuh"
#include "sm100.cuh"

namespace cslc {

using namespace sm100;

__device__ int g_page_decode_err = 0;

namespace {

constexpr int PD_THREADS = 192;
constexpr int PD_PROD_WARP = 4;
constexpr int PD_MMA_WARP = 5;
constexpr int PD_TILE = 128;
constexpr int PD_HALF = PD_TILE * 128;        // 16 KB: K or V codes of a tile
constexpr int PD_SMS = 148;
constexpr int PD_UNIT = 2;                    // what a unit costs besides its tiles, in tiles
constexpr int PD_WHOLE = 10;                  // tiles of a unit that one CTA takes alone, at most

enum { PD_ERR_EMPTY = 1, PD_ERR_K_FULL, PD_ERR_V_FULL, PD_ERR_Q_FULL, PD_ERR_Q_EMPTY, PD_ERR_S_FULL, PD_ERR_P_FULL,
       PD_ERR_O_FULL, PD_ERR_FINAL };

template <int STAGES>
struct __align__(8) PdBars {
  uint64_t k_full[STAGES], v_full[STAGES], empty[STAGES];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t q_full[2], q_empty[2], final_bar;
};

// Depth of the ring and buffers of q's parts, as shared memory allows for GP heads and PER CTAs
// of an SM. Two CTAs with three stages for pages of 32 tokens and more; three with two for pages
// of 16, whose many small copies leave a producer behind (8 x up to 131,072 tokens: 311 -> 251 us
// with pages of 16, but 229 -> 247 us with pages of 128).
constexpr int pd_stages(int per) { return per == 3 ? 2 : 3; }
constexpr int pd_qbufs(int gp) { return gp == 8 ? 2 : 1; }

template <int GP, int PER>
struct PdSmall {
  static constexpr int STAGES = pd_stages(PER);
  PdBars<STAGES> bars;
  float ks[STAGES][8];                     // scale of each page of the tile's keys
  int ev[STAGES][8];                       // exponent of its values' scale; PD_ABSENT: no such page
  __align__(16) float smax[2][GP][4];         // a tile's maxima by warp
  __align__(16) float lsum[2][GP][4];         // by segment parity
  float qs[pd_qbufs(GP)][GP];                            // what a score of the parts' products is multiplied with
  long long scan[PD_THREADS / 32];
  long long x_pre;                            // work before sequence x_b
  int x_b;
  uint32_t tmem_base;
  int abort_flag;
};

constexpr int PD_ABSENT = 1 << 20;

__device__ __forceinline__ float rcp_approx(float x) {   // within one unit in the last place
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
// Two values as two e4m3 parts each: x = hi + lo / 16, off by at most 2^-8 of x where hi is normal, 2^-14 below.
__device__ __forceinline__ void two_parts(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const float2 d = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3)));
  lo = __nv_cvt_float2_to_fp8x2(make_float2((a - d.x) * 16.f, (b - d.y) * 16.f), __NV_SATFINITE, __NV_E4M3);
}
// 2^d of a whole number d <= 0, 0 below 2^-126 and for NaN.
__device__ __forceinline__ float pow2i(float d) {
  return __uint_as_float((__float_as_uint(fmaxf(d, -127.f) + 12582912.f) << 23) + 0x3f800000u);
}

// A softmax warp's mbar_wait, out of line: inlined at each of its waits the code outgrew the instruction
// cache (64 requests of up to 8,192 tokens, pages of 128, 128 heads on 8: 130.9 against 118.2 us; 64 heads
// on 8: equal).
__device__ __noinline__ bool pd_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, int code) {
  return mbar_wait(bar, parity, abort, err, code);
}

struct PdShape {
  int B, H, Hkv, G, HG, page_log2, n_pages, max_pages, window;
  float scale_log2;
  long long q_stride;
  int whole;                                  // each CTA takes one unit, and all of it
};

// Visible tokens of sequence b: [lo, n); its tiles: [lo / 128, ceil(n / 128)).
__device__ __forceinline__ int pd_range(const PdShape& sh, const int32_t* __restrict__ seq_len, int b, int& lo, int& t0) {
  const long long cap = (long long)sh.max_pages << sh.page_log2;
  const int n = (int)min((long long)max(seq_len[b], 0), cap);
  lo = sh.window > 0 ? max(0, n - sh.window) : 0;
  t0 = lo / PD_TILE;
  return n;
}
__device__ __forceinline__ int pd_tiles(const PdShape& sh, const int32_t* __restrict__ seq_len, int b) {
  int lo, t0;
  const int n = pd_range(sh, seq_len, b, lo, t0);
  return n > 0 ? (n - 1) / PD_TILE + 1 - t0 : 0;
}

// Work of one unit of sequence b: its tiles and PD_UNIT, nothing without a tile.
__device__ __forceinline__ int pd_work(const PdShape& sh, const int32_t* __restrict__ seq_len, int b) {
  const int nt = pd_tiles(sh, seq_len, b);
  return nt > 0 ? nt + PD_UNIT : 0;
}

// Walks a CTA's range [x, x1) of the work, a segment (tiles of one unit) at a
// time. A unit's first PD_UNIT positions stand for its cost besides the tiles.
struct PdWalk {
  long long x, x1, pre;                       // pre: work before sequence b (over one unit each)
  int b;
  // the segment: tiles t .. t + len - 1 of the nt tiles of unit u of sequence b
  int u, t, len, nt;
  __device__ __forceinline__ bool next(const PdShape& sh, const int32_t* __restrict__ seq_len) {
    if (x >= x1) return false;
    const int HU = sh.Hkv * sh.HG;
    int w;
    while (true) {
      w = pd_work(sh, seq_len, b);
      if (x < (pre + w) * HU) break;
      pre += w;
      ++b;
    }
    nt = w - PD_UNIT;
    const long long off = x - pre * HU;
    u = (int)(off / w);
    const int r = (int)(off - (long long)u * w), skip = max(0, PD_UNIT - r);
    t = max(0, r - PD_UNIT);
    const long long most = x1 - x - skip;
    if (most <= 0) {                          // the range ends before the unit's first tile
      x = x1;
      return false;
    }
    len = (int)min((long long)(nt - t), most);
    x += skip + len;
    return true;
  }
};

}  // namespace

// Partials in the workspace: per CTA a header of 8 ints, then per slot (two per
// CTA: its first segment, its last one) GP x 128 sums and GP (reference, sum).
struct PdWs {
  int* hdr;       // [CTAs][8]: b, u, t, nt, work per CTA (two words); b = -1 when no unit continues here
  float* o;       // [2 CTAs][GP][128]
  float2* rl;     // [2 CTAs][GP]
};

template <int GP, int PER>
__global__ void __launch_bounds__(PD_THREADS, PER) page_decode_sm100_kernel(
    PdShape sh, const uint16_t* __restrict__ q, const float* __restrict__ k_scale, const float* __restrict__ v_scale,
    const int32_t* __restrict__ table, const int32_t* __restrict__ seq_len, uint16_t* __restrict__ out,
    float* __restrict__ lse, PdWs ws, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  constexpr int N = 2 * GP, QB = pd_qbufs(GP), STAGES = pd_stages(PER);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kv_s = smem;                                   // [STAGES][K 16 KB | V 16 KB]
  uint8_t* q_s = kv_s + STAGES * 2 * PD_HALF;          // [QB][N][128 B]
  uint8_t* p_s = q_s + QB * N * 128;                      // [2][N][128 B]
  PdSmall<GP, PER>* sm = reinterpret_cast<PdSmall<GP, PER>*>(p_s + 2 * N * 128);
  auto& bars = sm->bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int HU = sh.Hkv * sh.HG;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&bars.k_full[s], 1); mbar_init(&bars.v_full[s], 1); mbar_init(&bars.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1); mbar_init(&bars.p_full[i], 4); mbar_init(&bars.o_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) { mbar_init(&bars.q_full[i], 1); mbar_init(&bars.q_empty[i], 5); }
    mbar_init(&bars.final_bar, 1);
    sm->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == PD_MMA_WARP) tmem_alloc(&sm->tmem_base, 4 * N < 32 ? 32 : 4 * N);

  grid_dependency_wait();
  // ---- this CTA's range of the work: a scan over the sequences
  long long x0, x1, per = 0;
  if (sh.whole) {
    const int b = blockIdx.x / HU, w = pd_work(sh, seq_len, b);
    x0 = (long long)(blockIdx.x - b * HU) * w;            // counted from sequence b on
    x1 = x0 + w;
    if (tid == 0) { sm->x_pre = 0; sm->x_b = b; }
  } else {
    const int each = (sh.B + PD_THREADS - 1) / PD_THREADS;
    const int b0 = min(sh.B, tid * each), b1 = min(sh.B, b0 + each);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += pd_work(sh, seq_len, b);
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sm->scan[warp] = incl;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < PD_THREADS / 32; ++w) {
      if (w < warp) incl += sm->scan[w];
      total += sm->scan[w];
    }
    total *= HU;
    per = (total + gridDim.x - 1) / gridDim.x;
    x0 = min(total, per * blockIdx.x);
    x1 = min(total, x0 + per);
    // the thread whose sequences hold position x0 finds the sequence
    if (x0 < x1 && x0 >= (incl - sum) * HU && x0 < incl * HU) {
      long long pre = incl - sum;
      int b = b0;
      while (true) {
        const int w = pd_work(sh, seq_len, b);
        if (x0 < (pre + w) * HU) break;
        pre += w;
        ++b;
      }
      sm->x_pre = pre;
      sm->x_b = b;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  volatile int* abortp = &sm->abort_flag;
  int* errp = &g_page_decode_err;
  PdWalk walk;
  walk.x = x0; walk.x1 = x1; walk.pre = x0 < x1 ? sm->x_pre : 0; walk.b = x0 < x1 ? sm->x_b : 0;

  if (warp == PD_PROD_WARP) {
    // ------------------------------------------------------------ producer
    const int ppt = PD_TILE >> sh.page_log2;               // pages of a tile, at most 8
    const int P = 1 << sh.page_log2;
    if (lane == 0) { tma_prefetch_map(&tm_k); tma_prefetch_map(&tm_v); }
    int it = 0;
    // lane i < ppt holds page i of the tile: its first row (-1: there is none), its scales
    auto load = [&](int b, int u, int lo, int n, int tile, int& y, float& ks, float& vs) {
      y = -1; ks = vs = 0.f;
      if (lane < ppt) {
        const long long j = (long long)tile * ppt + lane;
        const long long tok = j << sh.page_log2;
        if (tok < n && tok + P > lo) {
          const int pid = table[(size_t)b * sh.max_pages + j];
          if (pid >= 0 && pid < sh.n_pages) {
            const int hk = u / sh.HG;
            const size_t ps = (size_t)pid * sh.Hkv + hk;
            y = (int)(ps << sh.page_log2);
            ks = k_scale[ps];
            vs = v_scale[ps];
          }
        }
      }
    };
    // q of a segment in two parts: lane = 4 dims, all heads' loads first
    auto put_q = [&](int seg, int b, int u) -> bool {
      const int qb = seg % QB;
      const int hk = u / sh.HG, g0 = (u - hk * sh.HG) * GP, gc = min(GP, sh.G - g0);
      const uint2* src = reinterpret_cast<const uint2*>(q + (long long)b * sh.q_stride + (hk * sh.G + g0) * kD) + lane;
      uint2 v[GP];
#pragma unroll
      for (int g = 0; g < GP; ++g) v[g] = g < gc ? src[g * (kD / 4)] : make_uint2(0u, 0u);
      bool w = true;
      if (seg >= QB) {
        if (lane == 0) w = mbar_wait(&bars.q_empty[qb], (uint32_t)((seg / QB - 1) & 1), abortp, errp, PD_ERR_Q_EMPTY);
        w = __shfl_sync(0xffffffffu, (int)w, 0) != 0;
        if (!w) return false;
      }
      uint8_t* dst = q_s + qb * N * 128;
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        const float f[4] = {bf16_lo(v[g].x), bf16_hi(v[g].x), bf16_lo(v[g].y), bf16_hi(v[g].y)};
        float am = 0.f;
        bool fin = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = fabsf(f[i]);
          fin = fin && a <= 3.402823466e38f;
          am = fmaxf(am, a <= 3.402823466e38f ? a : 0.f);
        }
        am = warp_redux_max(am);
        fin = __all_sync(0xffffffffu, fin);
        // am in [2^e, 2^(e+1)): times 2^(7 - e); the exponent is held where both powers are normal
        const int e = max(-110, (int)(__float_as_uint(am) >> 23) - 127) - 7;
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t hi = 0u, lw = 0u;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint32_t h2, l2;
          two_parts(f[i] * inv, f[i + 1] * inv, h2, l2);
          hi |= h2 << (8 * i);
          lw |= l2 << (8 * i);
        }
        *reinterpret_cast<uint32_t*>(dst + sw128(g, lane >> 2) + (lane & 3) * 4) = hi;
        *reinterpret_cast<uint32_t*>(dst + sw128(GP + g, lane >> 2) + (lane & 3) * 4) = lw;
        // a row of q that is not finite has no finite score
        const float back = __uint_as_float((uint32_t)(127 + e) << 23);
        if (lane == 0) sm->qs[qb][g] = fin ? sh.scale_log2 * back : __int_as_float(0x7fc00000);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_full[qb]);
      return true;
    };
    // the tiles of all segments in turn; a tile's page entries are loaded one tile ahead
    int lo = 0, n = 0, t0 = 0, i = 0, seg = -1;
    auto advance = [&]() -> bool {
      if (seg >= 0 && ++i < walk.len) return true;
      if (!walk.next(sh, seq_len)) return false;
      n = pd_range(sh, seq_len, walk.b, lo, t0);
      i = 0;
      ++seg;
      return true;
    };
    int y = -1;
    float ks = 0.f, vs = 0.f;
    bool more = advance();
    if (more) load(walk.b, walk.u, lo, n, t0 + walk.t, y, ks, vs);
    while (more) {
      const int s = it % STAGES;
      const bool new_seg = i == 0;
      const int seg_now = seg, b_now = walk.b, u_now = walk.u;
      int y2 = -1;
      float ks2 = 0.f, vs2 = 0.f;
      more = advance();
      if (more) load(walk.b, walk.u, lo, n, t0 + walk.t + i, y2, ks2, vs2);
      if (it >= STAGES) {
        bool w = true;
        if (lane == 0) w = mbar_wait(&bars.empty[s], (uint32_t)((it / STAGES - 1) & 1), abortp, errp, PD_ERR_EMPTY);
        if (!__shfl_sync(0xffffffffu, (int)w, 0)) break;
      }
      if (lane < ppt) {
        sm->ks[s][lane] = y >= 0 ? pow2(page_scale_exponent(ks)) : 0.f;
        sm->ev[s][lane] = y >= 0 ? page_scale_exponent(vs) : PD_ABSENT;
      }
      __syncwarp();
      if (lane == 0) { mbar_arrive_expect_tx(&bars.k_full[s], PD_HALF); mbar_arrive_expect_tx(&bars.v_full[s], PD_HALF); }
      __syncwarp();
      // a page that is not there reads the zero fill (a row past the end)
      if (lane < ppt) {
        const int row = y >= 0 ? y : max(1, (int)(((long long)sh.n_pages * sh.Hkv) << sh.page_log2));
        uint8_t* dst = kv_s + s * 2 * PD_HALF + (lane << sh.page_log2) * 128;
        tma_load_2d(dst, &tm_k, 0, row, &bars.k_full[s]);
        tma_load_2d(dst + PD_HALF, &tm_v, 0, row, &bars.v_full[s]);
      }
      ++it;
      if (new_seg && !put_q(seg_now, b_now, u_now)) break;
      y = y2; ks = ks2; vs = vs2;
    }
    // loads in flight after an abort land before the CTA leaves
    if (lane == 0)
      for (int d = 1; d <= STAGES && it - d >= 0; ++d) {
        const int k2 = it - d;
        mbar_wait_done(&bars.k_full[k2 % STAGES], (uint32_t)((k2 / STAGES) & 1), errp, PD_ERR_K_FULL);
        mbar_wait_done(&bars.v_full[k2 % STAGES], (uint32_t)((k2 / STAGES) & 1), errp, PD_ERR_V_FULL);
      }
    __syncwarp();
  } else if (warp == PD_MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t ID_S = idesc_e4m3(128, N);
      constexpr uint32_t ID_O = idesc_e4m3(128, N) | (1u << 15);   // A = V^T, MN-major
      int it = 0, seg = 0;
      bool ok = true;
      auto issue_pv = [&](int j) -> bool {
        const int s = j % STAGES, pb = j & 1;
        if (!mbar_wait(&bars.p_full[pb], (uint32_t)((j >> 1) & 1), abortp, errp, PD_ERR_P_FULL)) return false;
        if (!mbar_wait(&bars.v_full[s], (uint32_t)((j / STAGES) & 1), abortp, errp, PD_ERR_V_FULL)) return false;
        tc_fence_after();
        const uint32_t v0 = smem_u32(kv_s + s * 2 * PD_HALF + PD_HALF), p0 = smem_u32(p_s + pb * N * 128);
#pragma unroll
        for (int k = 0; k < 4; ++k)                                // 32 tokens each
          mma_e4m3(tmem + 2 * N + pb * N, smem_desc_sw128(v0 + k * 4096, PD_HALF, 1024),
                   smem_desc_sw128(p0 + k * 32, 16, 1024), ID_O, k > 0 ? 1u : 0u);
        mma_commit(&bars.o_full[pb]);
        mma_commit(&bars.empty[s]);
        return true;
      };
      while (ok && walk.next(sh, seq_len)) {
        const int qb = seg % QB;
        if (!mbar_wait(&bars.q_full[qb], (uint32_t)((seg / QB) & 1), abortp, errp, PD_ERR_Q_FULL)) break;
        const uint32_t q0 = smem_u32(q_s + qb * N * 128);
        ++seg;
        for (int i = 0; i < walk.len; ++i, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&bars.k_full[s], (uint32_t)((it / STAGES) & 1), abortp, errp, PD_ERR_K_FULL)) { ok = false; break; }
          tc_fence_after();
          const uint32_t k0 = smem_u32(kv_s + s * 2 * PD_HALF);
#pragma unroll
          for (int k = 0; k < 4; ++k)                              // 32 dims each
            mma_e4m3(tmem + (it & 1) * N, smem_desc_sw128(k0 + k * 32, 16, 1024), smem_desc_sw128(q0 + k * 32, 16, 1024),
                     ID_S, k > 0 ? 1u : 0u);
          mma_commit(&bars.s_full[it & 1]);
          if (i == walk.len - 1) mma_commit(&bars.q_empty[qb]);
          if (i > 0 && !issue_pv(it - 1)) { ok = false; break; }
        }
        if (ok && !issue_pv(it - 1)) ok = false;
      }
      mma_commit(&bars.final_bar);
      mbar_wait_done(&bars.final_bar, 0, errp, PD_ERR_FINAL);   // also after an abort: the products finish on their own
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const int pg = tid >> sh.page_log2;                   // this thread's page of a tile
    int it = 0;
    bool ok = true, w = true;
    // sequences without a visible token, spread over the CTAs
    for (int b = blockIdx.x; b < sh.B; b += gridDim.x)
      if (pd_tiles(sh, seq_len, b) == 0) {
        for (int h = 0; h < sh.H; ++h) out[((size_t)b * sh.H + h) * kD + tid] = 0;
        if (lse != nullptr && tid < sh.H) lse[(size_t)b * sh.H + tid] = -INFINITY;
      }
    if (tid == 0) {
      int* h = ws.hdr + 8 * blockIdx.x;
      h[0] = -1;
      h[4] = (int)(per & 0xffffffff);
      h[5] = (int)(per >> 32);
    }
    auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
      if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return;
      if (!__all_sync(0xffffffffu, pd_wait_slow(bar, parity, abortp, errp, code))) w = false;
    };
    auto load_cols = [&](uint32_t col, float (&x)[N]) {
#pragma unroll
      for (int c = 0; c < N; c += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + lane_off + col + c, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[c + i] = __uint_as_float(r[i]);
      }
    };
    int seg = 0;
    while (ok && walk.next(sh, seq_len)) {
      const int b = walk.b, hk = walk.u / sh.HG, g0 = (walk.u - hk * sh.HG) * GP;
      const int gc = min(GP, sh.G - g0);
      const size_t row0 = (size_t)b * sh.H + hk * sh.G + g0;
      int lo, t0;
      const int n = pd_range(sh, seq_len, b, lo, t0);
      const int qb = seg % QB;
      wait(&bars.q_full[qb], (uint32_t)((seg / QB) & 1), PD_ERR_Q_FULL);
      // The sums o and l are kept relative to 2^R, R the largest reference so far. References are
      // whole numbers, so that the factors between them are exponents. f: the last tile's factor.
      // Lanes 4 g .. 4 g + 3 hold R of head g (and of head 8 + g), and find the factors for all.
      constexpr int HL = GP / 8;
      float qs[GP], o[GP], l[GP], f[GP], R[HL];
#pragma unroll
      for (int g = 0; g < GP; ++g) { qs[g] = sm->qs[qb][g]; o[g] = 0.f; l[g] = 0.f; f[g] = 0.f; }
#pragma unroll
      for (int i = 0; i < HL; ++i) R[i] = -INFINITY;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_empty[qb]);
      auto join = [&](int j) {                            // tile j's O^T joins the sums
        wait(&bars.o_full[j & 1], (uint32_t)((j >> 1) & 1), PD_ERR_O_FULL);
        tc_fence_after();
        float x[N];
        load_cols(2 * N + (j & 1) * N, x);
        tmem_wait_ld();
#pragma unroll
        for (int g = 0; g < GP; ++g) o[g] = fmaf(f[g], fmaf(x[GP + g], 0.0625f, x[g]), o[g]);
      };
      for (int i = 0; i < walk.len; ++i, ++it) {
        const int s = it % STAGES, sb = it & 1;
        const int tok = (t0 + walk.t + i) * PD_TILE + tid;
        wait(&bars.k_full[s], (uint32_t)((it / STAGES) & 1), PD_ERR_K_FULL);   // the page's scales are there
        wait(&bars.s_full[sb], (uint32_t)((it >> 1) & 1), PD_ERR_S_FULL);
        tc_fence_after();
        float p[GP];
        const float ks = sm->ks[s][pg];
        const int ev = sm->ev[s][pg];
        const bool seen = tok >= lo && tok < n && ev != PD_ABSENT;
        {
          float x[N];
          load_cols(sb * N, x);
          const float evf = (float)ev;
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < GP; ++g) {
            const float sc = fmaf(x[GP + g], 0.0625f, x[g]) * ks;
            p[g] = seen ? fmaf(sc, qs[g], evf) : -INFINITY;
            const float mx = warp_redux_max(p[g]);
            if (lane == 0) sm->smax[sb][g][warp] = mx;
          }
        }
        if (i > 0) join(it - 1);                          // while the other warps' maxima arrive
        // all scores are read: one vote on the waits, which also publishes the maxima
        ok = !named_bar_or(1, 128, !w || *abortp != 0);
        if (!ok) break;
        const float einv = seen ? __uint_as_float((uint32_t)(127 - ev) << 23) : 0.f;
        uint8_t* pt = p_s + sb * N * 128 + (tid & 15);
        float ref[HL], fl[HL], al[HL];
        bool up = false;
#pragma unroll
        for (int k = 0; k < HL; ++k) {
          float mx = (&sm->smax[sb][8 * k][0])[lane];     // 8 heads x 4 warps
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // the tile's largest probability becomes 2^7 .. 2^8; no score at all leaves -inf. From 2^27 on the step of
          // fp32's is above 8 (a reference 16 below would make it 2^16, and e4m3 saturates): it becomes 1, and what is a
          // step or more below it, 2^-16, is lost: 127 of those are 2^-9 of the sum.
          const float r = ceilf(mx) - (fabsf(mx) < 134217728.f ? 8.f : 0.f), Rn = fmaxf(R[k], r);
          up = up || r > R[k];
          fl[k] = pow2i(r - Rn);
          al[k] = pow2i(R[k] - Rn);
          ref[k] = r == -INFINITY ? 0.f : r;
          R[k] = Rn;
        }
        if (__any_sync(0xffffffffu, up)) {                // rarely, after the first tiles
#pragma unroll
          for (int g = 0; g < GP; ++g) {
            const float a = __shfl_sync(0xffffffffu, al[g >> 3], 4 * (g & 7));
            o[g] *= a;
            l[g] *= a;
          }
        }
#pragma unroll
        for (int g = 0; g < GP; g += 2) {
          float pr[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            pr[k] = ex2_approx(p[g + k] - __shfl_sync(0xffffffffu, ref[g >> 3], 4 * ((g + k) & 7)));
            f[g + k] = __shfl_sync(0xffffffffu, fl[g >> 3], 4 * ((g + k) & 7));
            l[g + k] = fmaf(f[g + k], pr[k] * einv, l[g + k]);
          }
          uint32_t h2, l2;
          two_parts(pr[0], pr[1], h2, l2);
          const int ck = tid >> 4;
          pt[sw128(g, ck)] = (uint8_t)h2;
          pt[sw128(g + 1, ck)] = (uint8_t)(h2 >> 8);
          pt[sw128(GP + g, ck)] = (uint8_t)l2;
          pt[sw128(GP + g + 1, ck)] = (uint8_t)(l2 >> 8);
        }
        // a tile with tokens that are not seen: their stale V rows may hold NaN
        const int first = (t0 + walk.t + i) * PD_TILE;
        if (first < lo || first > n - PD_TILE) {
          wait(&bars.v_full[s], (uint32_t)((it / STAGES) & 1), PD_ERR_V_FULL);
          if (w && !seen) {
            uint4* row = reinterpret_cast<uint4*>(kv_s + s * 2 * PD_HALF + PD_HALF + tid * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[sb]);
      }
      if (!ok) break;
      join(it - 1);
      // ---- the segment's sums: l over the warp, halving the heads that a lane holds
#pragma unroll
      for (int h = GP / 2, m = 16; m > 0; m >>= 1) {
        if (h > 0) {
          const bool up = lane & m;
#pragma unroll
          for (int g = 0; g < h; ++g) {
            const float give = up ? l[g] : l[g + h], keep = up ? l[g + h] : l[g];
            l[g] = keep + __shfl_xor_sync(0xffffffffu, give, m);
          }
          h >>= 1;
        } else {
          l[0] += __shfl_xor_sync(0xffffffffu, l[0], m);
        }
      }
      constexpr int LB = GP == 8 ? 2 : 1;                 // lanes (1 << LB) that hold the same head
      if ((lane & ((1 << LB) - 1)) == 0) sm->lsum[seg & 1][lane >> LB][warp] = l[0];
      tc_fence_before();
      ok = !named_bar_or(1, 128, !w || *abortp != 0);
      if (!ok) break;
      const bool whole = walk.len == walk.nt;
      const int slot = 2 * blockIdx.x + (seg > 0 ? 1 : 0);
      // of head tid, which is a head of warp 0
      float Rt = __shfl_sync(0xffffffffu, R[0], 4 * (lane & 7)), lt = 0.f;
      if constexpr (HL == 2) {
        const float R1 = __shfl_sync(0xffffffffu, R[HL - 1], 4 * (lane & 7));
        if (lane & 8) Rt = R1;
      }
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        const float4 l4 = *reinterpret_cast<const float4*>(sm->lsum[seg & 1][g]);
        const float lg = (l4.x + l4.y) + (l4.z + l4.w);
        if (tid == g) lt = lg;
        if (!whole)
          ws.o[((size_t)slot * GP + g) * kD + tid] = o[g];
        else if (g < gc)
          out[(row0 + g) * kD + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(o[g] * (lg == 0.f ? 0.f : rcp_approx(lg))));
      }
      if (!whole) {
        if (tid < GP) ws.rl[(size_t)slot * GP + tid] = make_float2(Rt, lt);
      } else if (lse != nullptr && tid < gc) {
        lse[row0 + tid] = lt == 0.f ? -INFINITY : (Rt + log2f(lt)) * kLn2;
      }
      if (seg == 0 && walk.t > 0 && tid == 0) {
        int* h = ws.hdr + 8 * blockIdx.x;
        h[0] = b; h[1] = walk.u; h[2] = walk.t; h[3] = walk.nt;
      }
      ++seg;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == PD_MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 4 * N < 32 ? 32 : 4 * N);
  }
}

// CTA c merges the unit that crosses from CTA c - 1 into CTA c, if c is the
// first border inside it, for one head. Thread = dim; all partials' references
// and sums are loaded at once, and their rows eight at a time: the time is that
// of a few dependent loads, also for a sequence alone that every CTA has a part of.
template <int GP>
__global__ void __launch_bounds__(128) page_decode_combine_kernel(PdShape sh, PdWs ws, uint16_t* __restrict__ out,
                                                                  float* __restrict__ lse) {
  __shared__ float w[PD_SMS * 3];                         // factor of each partial
  grid_dependency_wait();
  const int c = blockIdx.x + 1, g = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int4 h = *reinterpret_cast<const int4*>(ws.hdr + 8 * c);   // b, u, t, nt
  const int2 h2 = *reinterpret_cast<const int2*>(ws.hdr + 8 * c + 4);
  const int b = h.x;
  if (b < 0) return;
  const long long per = ((long long)h2.y << 32) | (uint32_t)h2.x;
  const int u = h.y;
  const long long a = per * c - h.z, e = a + h.w;         // where the unit's tiles lie in the work
  const int c0 = (int)(a / per), n = (int)((e - 1) / per) - c0 + 1;
  if (c0 != c - 1) return;
  const int hk = u / sh.HG, g0 = (u - hk * sh.HG) * GP;
  if (g >= sh.G - g0) return;
  const int s0 = a - PD_UNIT <= per * c0 ? 2 * c0 : 2 * c0 + 1;   // the first segment of CTA c0, or its last
  auto at = [&](int k) { return (size_t)(k == 0 ? s0 : 2 * (c0 + k)) * GP + g; };
  // every warp finds the largest reference and the sum for itself
  float R = -INFINITY, l = 0.f;
  for (int k = lane; k < n; k += 32) R = fmaxf(R, ws.rl[at(k)].x);
  R = warp_redux_max(R);
  for (int k = lane; k < n; k += 32) {
    const float2 rl = ws.rl[at(k)];
    const float f = rl.x > -INFINITY && rl.x != R ? ex2_approx(rl.x - R) : 1.f;   // -inf: zeros, or NaN scores
    l = fmaf(rl.y, f, l);
    w[k] = f;                                             // the same value from each warp
  }
  l = warp_sum(l);
  __syncthreads();
  float o = 0.f;
#pragma unroll 8
  for (int k = 0; k < n; ++k) o = fmaf(ws.o[at(k) * kD + tid], w[k], o);
  const size_t row = (size_t)b * sh.H + hk * sh.G + g0 + g;
  out[row * kD + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(o * (l == 0.f ? 0.f : 1.f / l)));
  if (lse != nullptr && tid == 0) lse[row] = l == 0.f ? -INFINITY : (R + log2f(l)) * kLn2;
}

namespace {

// Query heads of one unit. Groups of up to 8 heads fill N = 16 columns; larger
// groups take 16 heads at a time (N = 32) and read the cache once for each 16.
int pd_group(int G) { return G <= 8 ? 8 : 16; }

template <int GP, int PER>
constexpr size_t pd_smem() {
  return 1024 + (size_t)pd_stages(PER) * 2 * PD_HALF + (pd_qbufs(GP) + 2) * 2 * GP * 128 + sizeof(PdSmall<GP, PER>);
}

template <int GP, int PER>
cslc_status pd_launch(PdShape sh, const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache,
                      const float* k_scale, const float* v_scale, const int32_t* table, const int32_t* seq_len,
                      uint16_t* out, float* lse, uint8_t* wsp, cudaStream_t stream) {
  cudaError_t err = cudaFuncSetAttribute(page_decode_sm100_kernel<GP, PER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)pd_smem<GP, PER>());
  if (err != cudaSuccess) return set_error(CSLC_ERR_CUDA, "cslc_page_decode_attn: %s", cudaGetErrorString(err));
  // an empty cache has no page to load; its map only has to be valid
  const uint64_t rows = (uint64_t)sh.n_pages * sh.Hkv << sh.page_log2;
  const void* kb = rows ? (const void*)k_cache : (const void*)q;
  const void* vb = rows ? (const void*)v_cache : (const void*)q;
  CUtensorMap tm_k, tm_v;
  if (!make_tmap_u8_rows128(&tm_k, kb, rows ? rows : 1, 1u << sh.page_log2) ||
      !make_tmap_u8_rows128(&tm_v, vb, rows ? rows : 1, 1u << sh.page_log2))
    return set_error(CSLC_ERR_CUDA, "cslc_page_decode_attn: tensor map encoding failed");
  PdWs ws;
  ws.hdr = reinterpret_cast<int*>(wsp);
  constexpr int most_ctas = PD_SMS * PER;
  ws.rl = reinterpret_cast<float2*>(wsp + most_ctas * 32);
  ws.o = reinterpret_cast<float*>(wsp + most_ctas * 32 + (size_t)2 * most_ctas * GP * sizeof(float2));
  const long long units = (long long)sh.B * sh.Hkv * sh.HG;
  const long long tokens = (long long)sh.max_pages << sh.page_log2;
  long long tiles = (tokens + PD_TILE - 1) / PD_TILE;     // of a unit, at most
  if (sh.window > 0 && sh.window < tokens) tiles = min(tiles, ((long long)sh.window + PD_TILE - 2) / PD_TILE + 1);
  // Units that are short at any length of their sequences go whole to a CTA each, which saves the
  // merge: 30 sequences of 8 key heads, window 512 / 1,024: 20.2 -> 14.2, 22.5 -> 17.6 us. Where
  // more of them than CTAs run at a time (64 sequences, window 1,024: 37.5 -> 40.7), or few longer ones
  // (16 units of 9 tiles: 11.4 -> 20.1), the even split is faster.
  sh.whole = units <= most_ctas && (tiles <= 4 || (tiles <= PD_WHOLE && units >= PD_SMS * 7 / 8));
  const long long most = sh.whole ? units : units * (tiles + PD_UNIT);
  const int grid = (int)(most < 1 ? 1 : most < most_ctas ? most : most_ctas);
  err = launch_after(page_decode_sm100_kernel<GP, PER>, dim3(grid), dim3(PD_THREADS), pd_smem<GP, PER>(), stream, sh, q,
                         k_scale, v_scale, table, seq_len, out, lse, ws, tm_k, tm_v);
  if (err != cudaSuccess) return set_error(CSLC_ERR_CUDA, "page_decode_sm100_kernel: %s", cudaGetErrorString(err));
  if (grid == 1 || sh.whole) return CSLC_OK;
  err = launch_after(page_decode_combine_kernel<GP>, dim3(grid - 1, sh.G < GP ? sh.G : GP), dim3(128), 0, stream, sh, ws,
                         out, lse);
  if (err != cudaSuccess) return set_error(CSLC_ERR_CUDA, "page_decode_combine_kernel: %s", cudaGetErrorString(err));
  return CSLC_OK;
}

}  // namespace

size_t page_decode_workspace_bytes(int, int H, int Hkv) {
  const int GP = pd_group(H / Hkv);
  const size_t ctas = PD_SMS * (GP == 8 ? 3 : 2);
  return ctas * 32 + 2 * ctas * GP * (sizeof(float2) + kD * sizeof(float));
}

cslc_status launch_page_decode(const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                               const float* v_scale, const int32_t* table, const int32_t* seq_len, int B, int H,
                               int Hkv, int page, int n_pages, int max_pages, long long q_stride, int window,
                               float scale, uint16_t* out, float* lse, void* ws, cudaStream_t stream) {
  const int G = H / Hkv, GP = pd_group(G);
  const PdShape sh{B, H, Hkv, G, (G + GP - 1) / GP, 31 - __builtin_clz(page), n_pages, max_pages, window,
                   scale * kLog2e, q_stride, 0};
  uint8_t* w = static_cast<uint8_t*>(ws);
  const auto run = GP == 16 ? pd_launch<16, 2> : page == 16 ? pd_launch<8, 3> : pd_launch<8, 2>;
  return run(sh, q, k_cache, v_cache, k_scale, v_scale, table, seq_len, out, lse, w, stream);
}

int page_decode_sm100_read_error() {
  int v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_page_decode_err, sizeof(int));
  if (v) cudaMemcpyToSymbol(g_page_decode_err, &zero, sizeof(int));
  return v;
}

CSLC_DEFINE_WAIT_LIMIT_SETTER(page_decode_sm100_set_wait_limits)

}  // namespace cslc
