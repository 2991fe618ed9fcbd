// Causal attention of packed sequences with grouped heads, on the 5th-generation
// tensor cores (tcgen05 + TMEM).
//
// Rows of a product are (token, head of the key head's group) pairs: with G
// heads to a key head a Q tile holds floor(128 / G) tokens. An item is two
// consecutive Q tiles of one sequence and key head; their keys and values are
// read once for both. Query i of a sequence sees the keys
// max(0, i + off - window + 1) .. i + off, off = nk - nq.
//
// CTA roles (persistent, one CTA per SM):
//   warps 0-3, 4-7  softmax and epilogue of Q tile 0 and 1, thread = row = TMEM
//                   lane. The row's reference is the maximum of its
//                   first visible tile and moves only when a tile's
//                   probabilities sum above 2^16 (O in TMEM is rescaled then),
//                   so the steady state needs no maximum; neither fp32 nor bf16
//                   loses precision to the larger numbers (values have to stay
//                   below 2^111 over the number of key tiles). P goes back to TMEM
//                   as bf16 (off by at most 2^-8 of itself) and is the A operand
//                   of P V from there: no shared memory and no proxy fence.
//   warp 8          producer: Q tiles (two items), K and V tiles of 64 keys
//                   (TMA, 6-deep ring of 16 KB); stores whole tiles of results
//   warps 9, 10     MMA issue for Q tile 0 and 1 (9 also allocates TMEM): S of
//                   the next tile as soon as this tile's scores are in
//                   registers, P V of this tile when P is there. So a softmax
//                   waits for neither product in the steady state.
// TMEM columns of a Q tile: S 64, P 2 x 32, O 128; both tiles fill the 512. A
// product S of 64 keys takes the pipe 48 cycles where half of one of 128 keys
// would take 32 (it is bound by reading Q and K), but with 128 keys P has to lie
// over S, and S of the next tile waits for P V of this one: 16.8 ms against 15.9.
//
// Measured (64 heads on 8, causal): 32,768 tokens 15.3-15.5 ms = 1,135-1,150 TFLOP/s
// at the power limit (1,665 MHz; cuBLAS sustains 1,387 there), 8,192 tokens 1.01-1.03
// ms. There the tensor-core pipe is busy 80 % of the cycles, the exponential pipe 61 %; without
// any softmax arithmetic the same loop reaches 1,228 TFLOP/s. Exponentials moved
// to the FMA pipe by a polynomial, single instead of packed fp32 operations, and
// one thread issuing the products were all slower: at the power limit every
// instruction counts.
//
// Order of work. prompt_schedule_kernel sorts the Q-tile pairs of all sequences
// by their number of key tiles, largest first; the CTAs draw tickets, so ragged
// and causal work evens out. The longer half of the pairs is drawn one key head
// after the other, so that its keys and values stay in L2; the shorter half of all
// heads comes last, longest first, and evens out what the long ones leave (all
// pairs head by head left the SMs busy 93 % of the time at 8,192 tokens: 1.08 ms
// against 1.00; all heads mixed 16.5 ms against 15.4 at 32,768). A CTA draws its next
// item late, with six key tiles left to load: 4,096 tokens of 32 heads 173 -> 156 us.
// Few items (at most one for each CTA)
// need no order and no ticket: that saves the schedule's 5 us.
//
// A value that is masked for some row of a tile may be NaN or infinite, and
// 0 * NaN would reach that row through the product. So the V tiles that are
// masked in part (about two for each Q tile) are scanned, and where one is not
// finite its P V is done on the CUDA cores, without the masked entries.
// All waits are time-bounded; no barrier without a bound is used in the loop.

#include "dependent.cuh"
#include "sm100.cuh"

namespace cslc {

using namespace sm100;

__device__ int g_prompt_attn_err = 0;

namespace {

constexpr int PA_THREADS = 352;
constexpr int PA_PROD_WARP = 8;
constexpr int PA_MMA_WARP = 9;
constexpr int PA_ROWS = 128;                     // rows of a Q tile
constexpr int PA_KEYS = 64;                      // keys of a K or V tile
constexpr int PA_SLOTS = 6;
constexpr int PA_Q_BYTES = PA_ROWS * 256;        // two halves of 64 dims
constexpr int PA_KV_BYTES = PA_KEYS * 256;
constexpr int PA_KV_HALF = PA_KEYS * 128;
constexpr float PA_SUM_MAX = 65536.f;            // of a tile: values of up to 2^111 / n do not overflow O over n key tiles
constexpr float PA_FAR = 4194304.f;              // 2^22: up to here m log2(e) scale is off by at most 1/4
constexpr int PA_SMS = 148;
constexpr int PA_APART = 450;                    // cycles between the Q tiles' softmaxes, in items of more
constexpr int PA_APART_MIN = 12;                 // key tiles than this
constexpr int PA_BUCKETS = 512;
constexpr int PA_SCHED_THREADS = 1024;

enum { PA_ERR_ITEM = 1, PA_ERR_Q_EMPTY, PA_ERR_EMPTY, PA_ERR_Q_FULL, PA_ERR_K_FULL, PA_ERR_V_FULL, PA_ERR_P_FULL,
       PA_ERR_O_FREE, PA_ERR_S_FULL, PA_ERR_S_READ, PA_ERR_PV_DONE, PA_ERR_O_FULL, PA_ERR_SLOW, PA_ERR_FINAL };

struct __align__(8) PaBars {
  uint64_t full[PA_SLOTS], empty[PA_SLOTS];
  uint64_t q_full[2], q_empty[2];                // by item parity
  uint64_t s_full[2], s_read[2], o_full[2], o_free[2], slow_done[2];   // by Q tile
  uint64_t p_full[2][2], pv_done[2][2];          // [Q tile][buffer]
  uint64_t item_full[2], item_empty[2];
  uint64_t final_bar[2];
};

struct PaShape {
  int B, Tq, Tk, H, Hkv, G, tpt, window;
  float scale, scale_log2;
  int direct;                                    // no schedule: CTA = item
};

// One item: two Q tiles of a sequence at its tokens t0 .. t0 + 2 tpt - 1.
struct PaItem {
  int q0, nq, k0, off, t0;                       // rows of q and k, nk - nq, first token of tile 0
  int n[2], s[2], e[2];                          // per Q tile: tokens, key tiles [s, e)
  int jb, je;
};

struct PaTake {
  int there, hk;                                 // an item, its key head; not there: no more
  PaItem it;
};

struct PaSmall {
  PaBars bars;
  PaTake take[2];                                // by item parity
  int bad_v[2][2];                               // [Q tile][buffer]: the last tile (from 1) whose V was not finite
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ void pa_seq(const PaShape& sh, const int32_t* __restrict__ cu_q,
                                       const int32_t* __restrict__ cu_k, int b, int& q0, int& nq, int& k0, int& nk) {
  q0 = min(max(cu_q[b], 0), sh.Tq);
  nq = min(max(cu_q[b + 1], q0), sh.Tq) - q0;
  k0 = min(max(cu_k[b], 0), sh.Tk);
  nk = min(max(cu_k[b + 1], k0), sh.Tk) - k0;
}

__device__ __forceinline__ PaItem pa_item(const PaShape& sh, const int32_t* __restrict__ cu_q,
                                          const int32_t* __restrict__ cu_k, int b, int pair) {
  PaItem it;
  int nk;
  pa_seq(sh, cu_q, cu_k, b, it.q0, it.nq, it.k0, nk);
  it.off = nk - it.nq;
  it.t0 = pair * 2 * sh.tpt;
  it.jb = 0x7fffffff;
  it.je = 0;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int tw = it.t0 + w * sh.tpt;
    it.n[w] = min(max(it.nq - tw, 0), sh.tpt);
    it.s[w] = it.e[w] = 0;
    const int last = tw + it.n[w] - 1 + it.off;  // the last token's last key
    if (it.n[w] > 0 && last >= 0) {
      it.e[w] = last / PA_KEYS + 1;
      it.s[w] = sh.window > 0 ? max(0, tw + it.off - sh.window + 1) / PA_KEYS : 0;
      it.jb = min(it.jb, it.s[w]);
      it.je = max(it.je, it.e[w]);
    }
  }
  if (it.je == 0) it.jb = 0;
  return it;
}

__device__ __forceinline__ int pa_pairs(const PaShape& sh, int nq) { return (nq + 2 * sh.tpt - 1) / (2 * sh.tpt); }

// D[tmem] (+)= A[tmem] * B[smem]^T (kind::f16, K = 16): bf16 A, two values to a column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
// The wait for 64 columns' values; they are tied to it, so that no use of them moves in front of it.
__device__ __forceinline__ void tmem_wait_ld64(uint32_t (&r)[2][32]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[0][i]), "+r"(r[1][i]));
}
// A box of shared memory into the tensor of `map`, and the waits for a thread's own stores: until
// they have read their source, and until they are done.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(map),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void bulk_store_commit() { asm volatile("cp.async.bulk.commit_group;\n" ::: "memory"); }
__device__ __forceinline__ void bulk_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void bulk_store_wait() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n" : "=r"(r) : "r"(taddr));
  return r;
}

// mbar_wait with the part that really waits out of line. The kernel's code competes for the instruction cache:
// a dozen inlined waits cost 3 % of 17 ragged prompts and 6 % of 100 short ones; unrolled staging cost 11 % of those.
__device__ __noinline__ bool pa_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, int code) {
  return mbar_wait(bar, parity, abort, err, code);
}
__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, int code) {
  return mbar_test(bar, parity) || pa_wait_slow(bar, parity, abort, err, code);
}
// Out of line: their registers and code stay out of the softmax loop's.
// A row of O (none of it: zeros) through 1 / l into its place of the Q tile, row -1: nothing.
__device__ __noinline__ void pa_stage_rows(uint32_t t_o, uint8_t* stage, int row, bool any, bool nothing, float inv) {
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    uint32_t r[32];
    if (any) {
      tmem_ld32(t_o + k * 32, r);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = 0u;
    }
    if (row >= 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t pk[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          pk[q] = pack_bf16x2(__uint_as_float(r[8 * i + 2 * q]) * inv, __uint_as_float(r[8 * i + 2 * q + 1]) * inv);
          pk[q] = nothing ? 0u : pk[q];                  // a row that sees nothing: probabilities 0, sums 0
        }
        *reinterpret_cast<uint4*>(stage + (k >> 1) * (PA_ROWS * 128) + sw128(row, (k & 1) * 4 + i)) =
            make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
    }
  }
}
__device__ __noinline__ void pa_rescale(uint32_t t_o, float alpha) {
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    uint32_t r[32];
    tmem_ld32(t_o + k * 32, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
    tmem_st32(t_o + k * 32, r);
  }
}
// O += P V on the CUDA cores over the keys k0 .. k1 - 1 of the tile, which the row sees; the products into O are done.
__device__ __noinline__ void pa_slow_pv(uint32_t t_o, uint32_t t_p, const uint8_t* v_s, int k0, int k1, bool first) {
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {                          // 32 dims at a time
    uint32_t r[32];
    if (!first) {
      tmem_ld32(t_o + k * 32, r);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = 0u;
    }
#pragma unroll 1
    for (int key = 0; key < PA_KEYS; ++key) {
      const uint32_t p2 = tmem_ld1(t_p + (key >> 1));
      tmem_wait_ld();
      const float p = (key & 1) ? bf16_hi(p2) : bf16_lo(p2);
      const uint8_t* vr = v_s + (k >> 1) * PA_KV_HALF;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 u = *reinterpret_cast<const uint4*>(vr + sw128(key, (k & 1) * 4 + q));
        const uint32_t u4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = q * 8 + 2 * i;
          if (key >= k0 && key < k1) {
            r[d] = __float_as_uint(fmaf(p, bf16_lo(u4[i]), __uint_as_float(r[d])));
            r[d + 1] = __float_as_uint(fmaf(p, bf16_hi(u4[i]), __uint_as_float(r[d + 1])));
          }
        }
      }
    }
    tmem_st32(t_o + k * 32, r);
  }
  tmem_wait_st();
}
// A warp's rows r0 .. r0 + 31 of a tile, those below `full`, from there to `dst` (the tile's first row).
// A whole tile is left to the producer's TMA.
__device__ __noinline__ void pa_store_rows(uint16_t* dst, const uint8_t* stage, int r0, int full, int G, int H, int inv_g) {
  if (PA_ROWS - full < G) return;
  const int lane = threadIdx.x & 31, c = lane & 15;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int r = r0 + 2 * i + (lane >> 4);
    if (r < full) {
      const int t = r * inv_g >> 16, h = r - t * G;
      *reinterpret_cast<uint4*>(dst + ((size_t)t * H + h) * kD + c * 8) =
          *reinterpret_cast<const uint4*>(stage + (c >> 3) * (PA_ROWS * 128) + sw128(r, c & 7));
    }
  }
}

}  // namespace

// The workspace: tickets drawn, number of pairs (16 bytes), then the pairs (b, index) in the order of work.
struct PaWs {
  int* head;
  int2* list;
  int cap;                                       // entries of the list
};

// One CTA: pairs of all sequences, counting sort by their key tiles, largest first.
__global__ void __launch_bounds__(PA_SCHED_THREADS) prompt_schedule_kernel(PaShape sh, const int32_t* __restrict__ cu_q,
                                                                           const int32_t* __restrict__ cu_k, PaWs ws) {
  extern __shared__ int pa_before[];             // [B + 1] pairs before sequence b
  __shared__ long long warp_sum_s[PA_SCHED_THREADS / 32];   // 64 bits: sequences that overlap count twice
  __shared__ int bucket[PA_BUCKETS];
  __shared__ int most_s;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");   // the attention's CTAs set up meanwhile
  grid_dependency_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int each = (sh.B + PA_SCHED_THREADS - 1) / PA_SCHED_THREADS;
  const int b0 = min(sh.B, tid * each), b1 = min(sh.B, b0 + each);
  long long sum = 0;
  int most = 0;
  for (int b = b0; b < b1; ++b) {
    int q0, nq, k0, nk;
    pa_seq(sh, cu_q, cu_k, b, q0, nq, k0, nk);
    sum += pa_pairs(sh, nq);
    most = max(most, (nk + PA_KEYS - 1) / PA_KEYS);
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum_s[warp] = incl;
  if (tid == 0) most_s = 0;
  for (int i = tid; i < PA_BUCKETS; i += PA_SCHED_THREADS) bucket[i] = 0;
  __syncthreads();
  atomicMax(&most_s, most);
  for (int w = 0; w < warp; ++w) incl += warp_sum_s[w];
  long long at = incl - sum;
  for (int b = b0; b < b1; ++b) {
    pa_before[b] = (int)min(at, 0x7fffffffll);
    int q0, nq, k0, nk;
    pa_seq(sh, cu_q, cu_k, b, q0, nq, k0, nk);
    at += pa_pairs(sh, nq);
  }
  if (b0 < sh.B && b1 == sh.B) pa_before[sh.B] = (int)min(at, 0x7fffffffll);
  __syncthreads();
  const int n = min(pa_before[sh.B], ws.cap);     // more only where cu_q is not ascending
  // bucket 0: the most key tiles (with a window never more than the window and a pair's tokens span)
  int top = most_s;
  if (sh.window > 0) top = min(top, (sh.window + 2 * sh.tpt) / PA_KEYS + 2);
  auto pair_of = [&](int i, int& b, int& pair) {
    int lo = 0, hi = sh.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pa_before[mid] <= i) lo = mid; else hi = mid;
    }
    b = lo;
    pair = i - pa_before[lo];
    const PaItem it = pa_item(sh, cu_q, cu_k, b, pair);
    return (int)((long long)max(0, top - (it.je - it.jb)) * (PA_BUCKETS - 1) / max(1, top));
  };
  for (int i = tid; i < n; i += PA_SCHED_THREADS) {
    int b, pair;
    atomicAdd(&bucket[pair_of(i, b, pair)], 1);
  }
  __syncthreads();
  if (warp == 0) {
    int c[PA_BUCKETS / 32], s = 0;
#pragma unroll
    for (int k = 0; k < PA_BUCKETS / 32; ++k) { c[k] = bucket[lane * (PA_BUCKETS / 32) + k]; s += c[k]; }
    int in = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += y;
    }
    in -= s;
#pragma unroll
    for (int k = 0; k < PA_BUCKETS / 32; ++k) { bucket[lane * (PA_BUCKETS / 32) + k] = in; in += c[k]; }
  }
  __syncthreads();
  for (int i = tid; i < n; i += PA_SCHED_THREADS) {
    int b, pair;
    const int k = pair_of(i, b, pair);
    ws.list[atomicAdd(&bucket[k], 1)] = make_int2(b, pair);
  }
  if (tid == 0) { ws.head[0] = 0; ws.head[1] = n; }
}

__global__ void __launch_bounds__(PA_THREADS, 1) prompt_attn_sm100_kernel(
    PaShape sh, const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k, PaWs ws, uint16_t* __restrict__ out,
    float* __restrict__ lse, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;                                   // [2 items][2 tiles][2 halves][128][128 B]
  uint8_t* ring = q_s + 4 * PA_Q_BYTES;                  // [SLOTS][2 halves][64][128 B]
  PaSmall* sm = reinterpret_cast<PaSmall*>(ring + PA_SLOTS * PA_KV_BYTES);
  PaBars& bars = sm->bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = sh.tpt * sh.G;                        // rows of a Q tile that hold a (token, head)

  if (tid == 0) {
    for (int s = 0; s < PA_SLOTS; ++s) { mbar_init(&bars.full[s], 1); mbar_init(&bars.empty[s], 2); }
    for (int w = 0; w < 2; ++w) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.p_full[w][i], 4); mbar_init(&bars.pv_done[w][i], 1);
      }
      mbar_init(&bars.s_full[w], 1); mbar_init(&bars.s_read[w], 4);
      mbar_init(&bars.o_full[w], 1); mbar_init(&bars.o_free[w], 4); mbar_init(&bars.slow_done[w], 4);
      mbar_init(&bars.q_full[w], 1); mbar_init(&bars.q_empty[w], 10);
      mbar_init(&bars.item_full[w], 1); mbar_init(&bars.item_empty[w], 10);
      mbar_init(&bars.final_bar[w], 1);
      sm->bad_v[w][0] = sm->bad_v[w][1] = 0;
    }
    sm->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == PA_MMA_WARP) tmem_alloc(&sm->tmem_base, 512);
  // rows of no (token, head) are never loaded: zeros, so that their scores are finite
  if (rows < PA_ROWS)
    for (int i = tid; i < 8 * (PA_ROWS - rows) * 8; i += PA_THREADS) {
      const int part = i / ((PA_ROWS - rows) * 8), r = i % ((PA_ROWS - rows) * 8);
      reinterpret_cast<uint4*>(q_s + part * (PA_ROWS * 128) + rows * 128)[r] = make_uint4(0u, 0u, 0u, 0u);
    }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();                                // the schedule, or what precedes the call
  const uint32_t tmem = sm->tmem_base;
  volatile int* abortp = &sm->abort_flag;
  int* errp = &g_prompt_attn_err;

  if (warp == PA_PROD_WARP) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_map(&tm_q); tma_prefetch_map(&tm_k); tma_prefetch_map(&tm_v);
      int kv = 0;                                        // tiles put into the ring
      int n = 0, q_loads = 0;
      bool ok = true;
      auto load_tile = [&](const CUtensorMap* map, int hk, int row) -> bool {
        const int s = kv % PA_SLOTS;
        if (kv >= PA_SLOTS &&
            !pa_wait(&bars.empty[s], (uint32_t)((kv / PA_SLOTS - 1) & 1), abortp, errp, PA_ERR_EMPTY))
          return false;
        uint8_t* dst = ring + s * PA_KV_BYTES;
        mbar_arrive_expect_tx(&bars.full[s], PA_KV_BYTES);
        tma_load_3d(dst, map, 0, hk, row, &bars.full[s]);
        tma_load_3d(dst + PA_KV_HALF, map, 64, hk, row, &bars.full[s]);
        ++kv;
        return true;
      };
      const int n_pairs = sh.direct ? 0 : ws.head[1];
      const long long n_items = (long long)n_pairs * sh.Hkv;
      const int n_long = n_pairs / 2;                    // pairs drawn head by head
      auto fetch = [&](bool first) -> PaTake {           // the next item
        PaTake t;
        int b = -1, pair = 0;
        if (sh.direct) {
          if (first) {                                   // item = CTA: the pair by a walk over the sequences
            pair = blockIdx.x / sh.Hkv;
            t.hk = blockIdx.x % sh.Hkv;
            for (int c = 0; c < sh.B; ++c) {
              int q0, nq, k0, nk;
              pa_seq(sh, cu_q, cu_k, c, q0, nq, k0, nk);
              const int p = pa_pairs(sh, nq);
              if (pair < p) { b = c; break; }
              pair -= p;
            }
          }
        } else {
          const long long i = atomicAdd(ws.head, 1);
          if (i < n_items) {
            long long p = i - (long long)n_long * sh.Hkv;
            if (p < 0) { p = i % n_long; t.hk = (int)(i / n_long); }
            else { t.hk = (int)(p % sh.Hkv); p = n_long + p / sh.Hkv; }
            const int2 bp = ws.list[p];
            b = bp.x;
            pair = bp.y;
          }
        }
        t.there = b >= 0;
        if (b >= 0) t.it = pa_item(sh, cu_q, cu_k, b, pair);
        return t;
      };
      // Whole Q tiles' results are stored from their place in the Q tile when that is to be loaded again, an
      // item later: the softmax warps' own stores took 2,300 of the 22,600 cycles of an item of ten key tiles.
      int o_tok[2], o_hk[2], o_n[2][2];                  // by item parity: first token, key head, tokens by Q tile
      auto store_out = [&](int i) -> bool {
        if (!pa_wait(&bars.q_empty[i & 1], (uint32_t)((i >> 1) & 1), abortp, errp, PA_ERR_Q_EMPTY)) return false;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int o = (i & 1) ? o_n[1][w] : o_n[0][w], hk = (i & 1) ? o_hk[1] : o_hk[0];
          if (o < sh.tpt) continue;
          const int tok = ((i & 1) ? o_tok[1] : o_tok[0]) + w * sh.tpt;
          const uint8_t* src = q_s + ((i & 1) * 2 + w) * PA_Q_BYTES;
          tma_store_3d(&tm_o, src, 0, hk * sh.G, tok);
          tma_store_3d(&tm_o, src + PA_ROWS * 128, 64, hk * sh.G, tok);
        }
        bulk_store_commit();
        return true;
      };
      PaTake next = fetch(true);
      for (;; ++n) {
        const PaTake t = next;
        if (n >= 2 && !pa_wait(&bars.item_empty[n & 1], (uint32_t)(((n >> 1) - 1) & 1), abortp, errp, PA_ERR_ITEM)) break;
        sm->take[n & 1] = t;
        mbar_arrive(&bars.item_full[n & 1]);
        if (!t.there) {
          if (n >= 2 && !store_out(n - 2)) break;
          if (n >= 1) store_out(n - 1);
          break;
        }
        const PaItem& it = t.it;
        const int hk = t.hk;
        if (n >= 2) {
          if (!store_out(n - 2)) break;
          bulk_store_wait_read();
        }
        if (n & 1) { o_tok[1] = it.q0 + it.t0; o_hk[1] = hk; o_n[1][0] = it.n[0]; o_n[1][1] = it.n[1]; }
        else { o_tok[0] = it.q0 + it.t0; o_hk[0] = hk; o_n[0][0] = it.n[0]; o_n[0][1] = it.n[1]; }
        q_loads = n + 1;
        mbar_arrive_expect_tx(&bars.q_full[n & 1], (uint32_t)(4 * rows * 128));
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int tok = it.q0 + it.t0 + w * sh.tpt;
          uint8_t* dst = q_s + ((n & 1) * 2 + w) * PA_Q_BYTES;
          tma_load_3d(dst, &tm_q, 0, hk * sh.G, tok, &bars.q_full[n & 1]);
          tma_load_3d(dst + PA_ROWS * 128, &tm_q, 64, hk * sh.G, tok, &bars.q_full[n & 1]);
        }
        // in the order of use: K0 K1 V0 K2 V1 .. The next item is looked up with the last tiles in front of it.
        if (it.jb < it.je) ok = load_tile(&tm_k, hk, it.k0 + it.jb * PA_KEYS);
        if (ok && it.jb + 1 < it.je) ok = load_tile(&tm_k, hk, it.k0 + (it.jb + 1) * PA_KEYS);
        bool fetched = false;
        for (int j = it.jb; j < it.je && ok; ++j) {
          ok = load_tile(&tm_v, hk, it.k0 + j * PA_KEYS);
          if (ok && j + 2 < it.je) ok = load_tile(&tm_k, hk, it.k0 + (j + 2) * PA_KEYS);
          if (!fetched && j > it.jb && j + 6 >= it.je) { next = fetch(false); fetched = true; }
        }
        if (!ok) break;
        if (!fetched) next = fetch(false);
      }
      bulk_store_wait();
      // loads in flight after an abort land before the CTA leaves
      for (int d = 1; d <= 2 && q_loads - d >= 0; ++d)
        mbar_wait_done(&bars.q_full[(q_loads - d) & 1], (uint32_t)(((q_loads - d) >> 1) & 1), errp, PA_ERR_Q_FULL);
      for (int d = 1; d <= PA_SLOTS && kv - d >= 0; ++d) {
        const int k2 = kv - d;
        mbar_wait_done(&bars.full[k2 % PA_SLOTS], (uint32_t)((k2 / PA_SLOTS) & 1), errp, PA_ERR_K_FULL);
      }
    }
    __syncwarp();
  } else if (warp >= PA_MMA_WARP) {
    // ------------------------------------------------- MMA issuer of Q tile w
    // The whole warp walks the loop and one elected lane (always the same) waits and issues: descriptors stay
    // in uniform registers (a lone thread took 77-88 cycles for a product of 64).
    constexpr uint32_t ID_S = idesc_bf16(PA_ROWS, PA_KEYS, false, false);
    constexpr uint32_t ID_O = idesc_bf16(PA_ROWS, 128, false, true);
    const int w = warp - PA_MMA_WARP;
    auto uni = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
    // low words of the descriptors of the Q tile and ring slot 0; an offset of x bytes adds x / 16
    const uint64_t d_kmaj = smem_desc_sw128(0, 16, 1024), d_mnmaj = smem_desc_sw128(0, PA_KV_HALF, 1024);
    const uint32_t r0 = smem_u32(ring) >> 4;
    const uint32_t t_s = uni(tmem + w * 128), t_o = uni(tmem + 256 + w * 128);
    int slot = 0, ph = 0;                                // the ring, in the order of use
    int s_it = 0, p_it = 0, o_it = 0, slow_it = 0;       // S and P tiles, items with a tile, tiles not done here
    // A lane's own, as giving up a wait is: around an abort one lane may see a phase complete and another the flag
    // or the limit. Such a lane issues nothing more but walks on with the others, through elections and shuffles, and
    // the warp leaves by the vote at the next item. (A vote behind each wait of the whole warp: 8,192 tokens
    // 1.00 -> 1.10 ms; waits of one lane: equal.)
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity, int code) {
      ok = ok && mbar_wait(bar, (uint32_t)(parity & 1), abortp, errp, code);
    };
    auto next_slot = [&]() { if (++slot == PA_SLOTS) { slot = 0; ph ^= 1; } };
    for (int n = 0;; ++n) {
      wait(&bars.item_full[n & 1], n >> 1, PA_ERR_ITEM);
      if (!__all_sync(0xffffffffu, ok)) break;
      const PaTake t = sm->take[n & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.item_empty[n & 1]);
      if (!t.there) break;
      const PaItem& it = t.it;
      const uint32_t q0 = uni(smem_u32(q_s + ((n & 1) * 2 + w) * PA_Q_BYTES) >> 4);
      const int js = uni(w == 0 ? it.s[0] : it.s[1]), je = uni(w == 0 ? it.e[0] : it.e[1]);
      const int jb = uni(it.jb), jend = uni(it.je);
      wait(&bars.q_full[n & 1], n >> 1, PA_ERR_Q_FULL);
      if (jb == jend) {
        if (elect_one() && ok) mma_commit(&bars.q_empty[n & 1]);
        __syncwarp();
      }
      auto issue_s = [&](int j) {
        const bool use = j >= js && j < je;
        const uint32_t lb = uni(r0 + slot * (PA_KV_BYTES / 16));
        if (elect_one()) {
          wait(&bars.full[slot], ph, PA_ERR_K_FULL);
          if (use && s_it > 0) wait(&bars.s_read[w], s_it - 1, PA_ERR_S_READ);   // the last scores are in registers
          if (ok) {
            if (use) {
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma_bf16(t_s, d_kmaj | (q0 + ((k >> 2) * (PA_ROWS * 128) + (k & 3) * 32) / 16),
                         d_kmaj | (lb + ((k >> 2) * PA_KV_HALF + (k & 3) * 32) / 16), ID_S, k > 0 ? 1u : 0u);
              mma_commit(&bars.s_full[w]);
            }
            mma_commit(&bars.empty[slot]);               // (or it is the other Q tile's alone)
            if (j == jend - 1) mma_commit(&bars.q_empty[n & 1]);   // every S of the item has read Q
          }
        }
        __syncwarp();
        if (use) ++s_it;
        next_slot();
      };
      if (jb < jend) issue_s(jb);
      for (int j = jb; j < jend; ++j) {
        if (j + 1 < jend) issue_s(j + 1);
        const bool use = j >= js && j < je, first = j == js;
        const int b = p_it & 1;
        const uint32_t lo = uni(r0 + slot * (PA_KV_BYTES / 16)), a = uni(t_s + 64 + b * 32);
        if (elect_one()) {
          wait(&bars.full[slot], ph, PA_ERR_V_FULL);
          if (use) {
            if (first && o_it > 0) wait(&bars.o_free[w], o_it - 1, PA_ERR_O_FREE);
            wait(&bars.p_full[w][b], p_it >> 1, PA_ERR_P_FULL);
            // a V tile that is not finite where some row does not see it: the softmax warps did the product
            const bool mine = reinterpret_cast<volatile int*>(sm->bad_v[w])[b] != p_it + 1;
            if (!mine) wait(&bars.slow_done[w], slow_it++, PA_ERR_SLOW);
            if (ok) {
              tc_fence_after();
              if (mine) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_bf16_ts(t_o, a + k * 8, d_mnmaj | (lo + k * (2048 / 16)), ID_O, (!first || k > 0) ? 1u : 0u);
              }
              mma_commit(&bars.pv_done[w][b]);
              if (j == je - 1) mma_commit(&bars.o_full[w]);
            }
          }
          if (ok) mma_commit(&bars.empty[slot]);
        }
        __syncwarp();
        if (use) { ++p_it; if (first) ++o_it; }
        next_slot();
      }
    }
    if (elect_one()) mma_commit(&bars.final_bar[w]);
    __syncwarp();
    mbar_wait_done(&bars.final_bar[w], 0, errp, PA_ERR_FINAL);   // also after an abort: the products finish on their own
    __syncwarp();
  } else {
    // ------------------------------------------------------ softmax + epilogue
    const int w = warp >> 2;
    const int row = tid & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + w * 128, t_o = tmem + lane_off + 256 + w * 128;
    const float c = sh.scale_log2;
    int kv0 = 0, t_it = 0, o_it = 0;                     // ring position, this Q tile's key tiles, items
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity, int code) -> bool {
      if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abortp, errp, code));
    };
    auto wait_out = [&](uint64_t* bar, uint32_t parity, int code) -> bool {
      if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
      return __all_sync(0xffffffffu, pa_wait_slow(bar, parity, abortp, errp, code));
    };
    // is the V tile at ring position vv finite? Two threads to a key; a warp finds out about its 16
    auto scan_v = [&](int vv, bool& bad) -> bool {
      const int vs = vv % PA_SLOTS, key = row >> 1;
      const uint8_t* v_s = ring + vs * PA_KV_BYTES + (row & 1) * PA_KV_HALF + key * 128;
      if (!wait(&bars.full[vs], (uint32_t)((vv / PA_SLOTS) & 1), PA_ERR_V_FULL)) return false;
      uint32_t ones = 0u;                                // an exponent of all ones carries into the sign's place
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint4 u = *reinterpret_cast<const uint4*>(v_s + ((k ^ (key & 7)) << 4));
        const uint32_t u4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) ones |= ((u4[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
      }
      bad = __any_sync(0xffffffffu, ones != 0u);
      return true;
    };
    const int ti = row / sh.G, inv_g = 65535 / sh.G + 1; // this row's token of the Q tile; r / G = r inv_g >> 16
    for (int n = 0; ok; ++n) {
      if (!wait_out(&bars.item_full[n & 1], (uint32_t)((n >> 1) & 1), PA_ERR_ITEM)) break;
      if (!sm->take[n & 1].there) break;
      const PaItem& it = sm->take[n & 1].it;             // stays there until the tile is done
      const int tw = it.t0 + w * sh.tpt;                 // the Q tile's first token
      const int j0 = it.s[w], j1 = it.e[w];
      const int tok = tw + ti;                           // this row's token
      const bool row_ok = ti < it.n[w];
      const int last = tok + it.off;                     // its last key (below 0: none) and first
      const int lo = sh.window > 0 ? max(0, last - sh.window + 1) : 0;
      // tiles masked for no token of the Q tile: [whole0, whole1)
      const int whole0 = sh.window > 0 ? (max(0, tw + it.n[w] - 1 + it.off - sh.window + 1) + PA_KEYS - 1) / PA_KEYS : 0;
      const int whole1 = (tw + it.off + 1) / PA_KEYS;
      // The reference is M = c m rounded to fp32, the same number wherever it is used. Where that rounding could
      // move the row's largest probability far from 1 (up to 2^22 by a factor of at most 2^(1/4), from 2^31 on out of
      // fp32's range) it is c m itself, and c (s - m) is computed from the difference.
      bool far = false;                                  // such a row is in the warp
      float m = -INFINITY, l = 0.f;
      auto is_far = [&](float x) { return fabsf(x * c) > PA_FAR; };
      for (int j = j0; j < j1; ++j, ++t_it) {
        const int b = t_it & 1;
        const uint32_t t_p = t_s + 64 + b * 32;
        const bool part = j < whole0 || j >= whole1;
        // ring position of its V: behind the K of up to two tiles more
        auto vv = [&]() { return kv0 + (j - it.jb) + min(j - it.jb + 2, it.je - it.jb); };
        if (!wait_out(&bars.s_full[w], (uint32_t)(t_it & 1), PA_ERR_S_FULL)) { ok = false; break; }
        // (the PV of two tiles before, which read this tile's P buffer, was issued before these
        // scores, so it is done too)
        tc_fence_after();
        // An item's two softmaxes keep the distance that they start with, and run best a third of a tile apart,
        // where one loads scores while the other has the exponentials: 8,192 tokens 1.077 ms with 200 cycles,
        // 1.013 with 400 to 500, 1.022 with 600, 1.05 with 0 or 900. A short item would not earn the wait.
        if (w == 0 && j == j0 && j1 - j0 > PA_APART_MIN) {
          const long long t0 = clock64();
          while (clock64() - t0 < PA_APART) {}
        }
        uint32_t s[2][32];
        auto at = [&](int k) { return __uint_as_float(s[k >> 5][k & 31]); };
        tmem_ld32(t_s, s[0]);
        tmem_ld32(t_s + 32, s[1]);
        tmem_wait_ld64(s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.s_read[w]);
        if (part) {
          const int hi = row_ok ? last + 1 - j * PA_KEYS : PA_KEYS, l0 = row_ok ? lo - j * PA_KEYS : 0;
          // one select for each key, by a bit: two passes of compares were 2 to 3 % slower in all
          const uint64_t seen = (hi >= 64 ? ~0ull : hi <= 0 ? 0ull : (1ull << hi) - 1) & (l0 <= 0 ? ~0ull : l0 >= 64 ? 0ull : ~0ull << l0);
          const uint32_t seen2[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
#pragma unroll
          for (int k = 0; k < 64; ++k) s[k >> 5][k & 31] = (seen2[k >> 5] & (1u << (k & 31))) ? s[k >> 5][k & 31] : 0xff800000u;
        }
        auto row_max = [&]() -> float {
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = at(k);
#pragma unroll
          for (int k = 4; k < 64; ++k) mx[k & 3] = fmaxf(mx[k & 3], at(k));
          return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        };
        if (__any_sync(0xffffffffu, m == -INFINITY)) {   // the row's first visible keys set the reference
          if (m == -INFINITY) m = row_max();
          far = __any_sync(0xffffffffu, is_far(m) && m != -INFINITY);
        }
        // P = 2^(c s - M) as bf16, two to a column
        const float neg = m == -INFINITY ? 0.f : -__fmul_rn(m, c);
        float2 ps[4];
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 4; ++k) ps[k] = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float2 a = fma2(make_float2(at(2 * k), at(2 * k + 1)), make_float2(c, c), make_float2(neg, neg));
          a = make_float2(ex2_approx(a.x), ex2_approx(a.y));
          ps[k & 3] = add2(ps[k & 3], a);
          pk[k] = pack_bf16x2(a.x, a.y);
        }
        ps[0] = add2(add2(ps[0], ps[1]), add2(ps[2], ps[3]));
        float sum = ps[0].x + ps[0].y;
        // a stale reference (the probabilities leave the range), or a far one: the warp redoes the tile
        const bool over = !(sum <= PA_SUM_MAX), redo = __any_sync(0xffffffffu, over) || far;
        auto last_pv_done = [&]() -> bool {
          if (j == j0) return true;
          const bool y = wait(&bars.pv_done[w][b ^ 1], (uint32_t)(((t_it - 1) >> 1) & 1), PA_ERR_PV_DONE);
          tc_fence_after();
          return y;
        };
        if (redo) {
          if (!last_pv_done()) { ok = false; break; }
          const float mx = over ? fmaxf(row_max(), m) : m;
          // 2^(old reference - new one); probabilities are 2^((s - base) c + neg2)
          const bool was_far = is_far(m), now_far = is_far(mx);
          const float base = now_far && mx != -INFINITY ? mx : 0.f, neg2 = now_far ? 0.f : -__fmul_rn(mx, c);
          const float up = was_far ? fmaf(m - base, c, neg2) : now_far ? fmaf(-mx, c, __fmul_rn(m, c))
                                                                      : __fadd_rn(neg2, __fmul_rn(m, c));
          const float alpha = mx > m ? ex2_approx(up) : 1.f;
          m = mx;
          l *= alpha;
          far = __any_sync(0xffffffffu, now_far && m != -INFINITY);
          if (j > j0) pa_rescale(t_o, alpha);
          sum = 0.f;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float e0 = ex2_approx(fmaf(at(2 * k) - base, c, neg2)), e1 = ex2_approx(fmaf(at(2 * k + 1) - base, c, neg2));
            sum += e0 + e1;
            pk[k] = pack_bf16x2(e0, e1);
          }
        }
        l += sum;
        tmem_st32(t_p, pk);
        tmem_wait_st();
        if (part) {
          // now, not before: the tile's scores say that the ring is less than a turn before its V
          bool bad;
          if (!scan_v(vv(), bad)) { ok = false; break; }
          if (bad && lane == 0) reinterpret_cast<volatile int*>(sm->bad_v[w])[b] = t_it + 1;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[w][b]);
        if (part) {                                      // what the other warps found
          if (!wait(&bars.p_full[w][b], (uint32_t)((t_it >> 1) & 1), PA_ERR_P_FULL)) { ok = false; break; }
          if (reinterpret_cast<volatile int*>(sm->bad_v[w])[b] == t_it + 1) {
            if (!last_pv_done()) { ok = false; break; }
            pa_slow_pv(t_o, t_p, ring + (vv() % PA_SLOTS) * PA_KV_BYTES, lo - j * PA_KEYS, last + 1 - j * PA_KEYS, j == j0);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.slow_done[w]);
          }
        }
      }
      if (!ok) break;
      kv0 += 2 * (it.je - it.jb);
      // ---- epilogue
      const bool any = j1 > j0;
      // (without a key tile: the Q tile has landed)
      if (!(any ? wait_out(&bars.o_full[w], (uint32_t)(o_it++ & 1), PA_ERR_O_FULL)
                : wait_out(&bars.q_full[n & 1], (uint32_t)((n >> 1) & 1), PA_ERR_Q_FULL)))
        break;
      tc_fence_after();
      // The warp's 32 rows go through the item's Q tile, which every S has read, so that the stores are whole
      // rows (16 bytes of 32 rows in one store took 4,100 to 5,200 cycles an item) or the producer's.
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint8_t* stage = q_s + ((n & 1) * 2 + w) * PA_Q_BYTES;
      pa_stage_rows(t_o, stage, row < rows ? row : -1, any, l == 0.f, inv);
      if (row_ok && lse != nullptr)
        lse[(size_t)(it.q0 + tok) * sh.H + sm->take[n & 1].hk * sh.G + (row - ti * sh.G)] =
            l == 0.f ? -INFINITY : fmaf(m, sh.scale, (log2f(l) - (is_far(m) ? 0.f : fmaf(m, c, -__fmul_rn(m, c)))) * kLn2);
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.o_free[w]);
      }
      __syncwarp();
      pa_store_rows(out + ((size_t)(it.q0 + tw) * sh.H + sm->take[n & 1].hk * sh.G) * kD, stage, row & ~31, it.n[w] * sh.G, sh.G,
                    sh.H, inv_g);
      fence_proxy_async_smem();                          // the next Q tile lands where the rows were
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.item_empty[n & 1]);
        mbar_arrive(&bars.q_empty[n & 1]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == PA_MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {

// Q-tile pairs of all sequences at most: a pair for every 2 tpt tokens and one more for each sequence.
long long pa_most_pairs(int B, int Tq, int tpt) { return (long long)Tq / (2 * tpt) + (B < Tq ? B : Tq); }

// At most one item for each SM: no schedule. (The walk over the sequences is short then.)
bool pa_direct(int B, int Tq, int H, int Hkv) {
  return B <= PA_SMS && pa_most_pairs(B, Tq, PA_ROWS / (H / Hkv)) * Hkv <= PA_SMS;
}

}  // namespace

size_t prompt_attn_workspace_bytes(int B, int Tq, int H, int Hkv) {
  if (pa_direct(B, Tq, H, Hkv)) return 0;
  return 16 + (size_t)pa_most_pairs(B, Tq, PA_ROWS / (H / Hkv)) * sizeof(int2);
}

cslc_status launch_prompt_attn(const uint16_t* q, const uint16_t* k, const uint16_t* v, const int32_t* cu_q,
                               const int32_t* cu_k, int B, int Tq, int Tk, int H, int Hkv, long long q_stride,
                               long long k_stride, long long v_stride, int window, float scale, uint16_t* out,
                               float* lse, void* wsp, cudaStream_t stream) {
  const char* fn = "cslc_prompt_attn";
  if (window >= Tk) window = 0;                  // hides no key; differences with it stay within 32 bits
  const size_t smem = 1024 + 4 * PA_Q_BYTES + (size_t)PA_SLOTS * PA_KV_BYTES + sizeof(PaSmall);
  cudaError_t err = cudaFuncSetAttribute(prompt_attn_sm100_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return set_error(CSLC_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(err));
  const int G = H / Hkv, tpt = PA_ROWS / G;
  const long long items = pa_most_pairs(B, Tq, tpt) * Hkv;
  const PaShape sh{B, Tq, Tk, H, Hkv, G, tpt, window, scale, scale * kLog2e, pa_direct(B, Tq, H, Hkv) ? 1 : 0};
  CUtensorMap tm_q, tm_k, tm_v, tm_o;
  // without keys no tile of them is loaded: the maps only have to be valid
  const bool keys = Tk > 0;
  if (!make_tmap_bf16_rows128(&tm_q, q, H, Tq, q_stride, G, tpt) ||
      !make_tmap_bf16_rows128(&tm_k, keys ? k : q, keys ? Hkv : H, keys ? Tk : Tq, keys ? k_stride : q_stride, 1, PA_KEYS) ||
      !make_tmap_bf16_rows128(&tm_o, out, H, Tq, (long long)H * kD, G, tpt) ||
      !make_tmap_bf16_rows128(&tm_v, keys ? v : q, keys ? Hkv : H, keys ? Tk : Tq, keys ? v_stride : q_stride, 1, PA_KEYS))
    return set_error(CSLC_ERR_CUDA, "%s: tensor map encoding failed", fn);
  PaWs ws;
  ws.head = static_cast<int*>(wsp);
  ws.list = reinterpret_cast<int2*>(static_cast<uint8_t*>(wsp) + 16);
  ws.cap = (int)pa_most_pairs(B, Tq, tpt);
  if (!sh.direct) {
    err = launch_after(prompt_schedule_kernel, dim3(1), dim3(PA_SCHED_THREADS), (size_t)(B + 1) * sizeof(int), stream, sh,
                           cu_q, cu_k, ws);
    if (err != cudaSuccess) return set_error(CSLC_ERR_CUDA, "prompt_schedule_kernel: %s", cudaGetErrorString(err));
  }
  err = launch_after(prompt_attn_sm100_kernel, dim3((unsigned)(items < PA_SMS ? items : PA_SMS)), dim3(PA_THREADS), smem,
                         stream, sh, cu_q, cu_k, ws, out, lse, tm_q, tm_k, tm_v, tm_o);
  if (err != cudaSuccess) return set_error(CSLC_ERR_CUDA, "prompt_attn_sm100_kernel: %s", cudaGetErrorString(err));
  return CSLC_OK;
}

int prompt_attn_sm100_read_error() {
  int v = 0, zero = 0;
  cudaMemcpyFromSymbol(&v, g_prompt_attn_err, sizeof(int));
  if (v) cudaMemcpyToSymbol(g_prompt_attn_err, &zero, sizeof(int));
  return v;
}

CSLC_DEFINE_WAIT_LIMIT_SETTER(prompt_attn_sm100_set_wait_limits)

}  // namespace cslc
