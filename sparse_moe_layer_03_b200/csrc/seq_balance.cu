// The balance loss over packed sequences ("MOE-DIT", eq. L_balance, whose T is the
// length of one image-patch sequence): its per-sequence expert counts, its value and,
// joined with the gates' gradient, its gradient through the router.
//
// Sequence b holds rows off[b] .. off[b+1]-1, L_b of them, and c[b,i] of their selected
// pairs are expert i's.  With P the router's scores and B' the sequences that hold a row,
//     loss_b = alpha sum_i E / (K L_b) c[b,i] 1/L_b sum_{t in b} P[t,i],   L = 1/B' sum_b loss_b
//     dP[t,i] = aux_scale alpha E c[b,i] / (K L_b^2 B') + dgate on the selected slots
//     dl = P (dP - sum_j P dP),   dWg = dl^T x,   db = sum_t dl,   dx (+)= dl Wg.
// A token's share of its sequence's loss, sum_i P[t,i] C[b,i] with C = alpha E c / (K L_b^2),
// is a by-product of the softmax's backward.  Rows of no sequence take no part: their x is
// not read (whatever it holds) and their dx stays.
//
// Four launches, each bound by memory, none with a barrier in its loop:
//   count   sequence and factor of every token, counts (integer atomics)
//   scores  logits, softmax, dl: reads x once
//   grads   dx and the partial sums of dWg: reads x again (from L2 where it fits), dx in and out
//   finish  the partial sums of dWg and db in a fixed order, the losses
// They are chained by programmatic dependent launch: scores forms its logits while count runs.
//
// The 16-bit kernels take their operands straight from global memory into mma.sync fragments.
// Where an index is summed over (the columns in the logits) or names an output (the columns of dx
// and of dWg) the order in which a fragment holds it is free, so each lane's fragments are chosen
// to be 16 consecutive bytes of a row: no shared memory, no ldmatrix, full sectors.  dWg sums over
// tokens, whose pairs lie in different rows: two rows' 16-byte vectors are interleaved in registers.
// dl goes between the kernels already in fragment order, as it is and transposed (movmatrix), in
// two 16-bit parts hi + lo (bf16: 16 bits of mantissa; fp16: 22 bits below its row's, or its
// 16-token block's, largest).  With E <= 8 both parts share one k16 step.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kCountThreads = 256;
constexpr int kOffSmem = 2048;                     // offsets kept in shared memory up to this many
constexpr int kFinThreads = 256;

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
// first and one past the last row that belong to a sequence
__device__ __forceinline__ void live_rows(const SeqBalArgs& a, int& lo, int& hi) {
  lo = a.offsets ? min(max(a.offsets[0], 0), a.T) : 0;
  hi = a.offsets ? min(max(a.offsets[a.n_seqs], lo), a.T) : a.T;
}
__device__ __forceinline__ int slots_of(const SeqBalArgs& a, int t) {
  return a.n_sel ? min(max(a.n_sel[t], 0), a.Kmax) : a.K;
}

// ---------------------------------------------------------------- count
// One thread per token: its sequence by binary search, its selected experts into the counts (equal
// (sequence, expert) keys of a warp merged first, as in the frequency kernel).
__global__ void __launch_bounds__(kCountThreads) seq_count_kernel(SeqBalArgs a) {
  __shared__ int off_s[kOffSmem];
  launch_dependents();
  const int tid = threadIdx.x, n = a.n_seqs;
  const int* off = a.offsets;
  if (off) {
    const bool in_smem = n + 1 <= kOffSmem;
    if (in_smem) {
      for (int i = tid; i <= n; i += kCountThreads) off_s[i] = off[i];
      __syncthreads();
      off = off_s;
    }
    int full = 0;                                  // this block's share of the sequences
    for (int b = blockIdx.x * kCountThreads + tid; b < n; b += gridDim.x * kCountThreads) {
      const int lo = off[b], hi = off[b + 1];
      if (lo < 0 || hi < lo || hi > a.T) set_status(a.status, DEV_BAD_INDEX, 410);
      full += hi > lo;
    }
    full = __reduce_add_sync(0xffffffffu, full);
    if ((tid & 31) == 0 && full) atomicAdd(a.live, full);
  } else if (blockIdx.x == 0 && tid == 0) {
    *a.live = n;
  }
  const int t = blockIdx.x * kCountThreads + tid;
  int sid = -1, len = 0;
  if (t < a.T) {
    if (off) {
      int lo = 0, hi = n;                          // the last sequence that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= t) lo = mid + 1;
        else hi = mid;
      }
      sid = lo - 1;
      if (sid >= 0) {
        len = off[sid + 1] - off[sid];
        if (t < off[sid] || t >= off[sid + 1]) sid = -1;   // (the first holds where offsets descend)
      }
    } else {
      sid = t / a.seq_len;
      len = a.seq_len;
    }
    const float coef = sid >= 0 ? (float)((double)a.alpha * a.E / ((double)a.K * len * len)) : 0.f;
    a.tok[t] = make_int2(sid, __float_as_int(coef));
  }
  const int ns = sid >= 0 ? slots_of(a, t) : 0;
  for (int k = 0; k < a.Kmax; ++k) {
    long long key = -1;
    if (k < ns) {
      const int e = a.topk_idx[(size_t)t * a.Kmax + k];
      if (e >= a.E) set_status(a.status, DEV_BAD_INDEX, 411);
      else if (e >= 0) key = (long long)sid * a.E + e;
    }
    const unsigned same = __match_any_sync(0xffffffffu, key);
    if (key >= 0 && (tid & 31) == __ffs(same) - 1) atomicAdd(&a.counts[key], __popc(same));
  }
}

// ---------------------------------------------------------------- scores, 16-bit types
template <bool F16> struct H16;
template <> struct H16<false> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
};
template <> struct H16<true> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_f16x2(lo, hi); }
  static __device__ __forceinline__ float2 unpack(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
};
__device__ __forceinline__ uint32_t movm_t(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// power of two that brings m into [1, 2) (1 for 0 and for what has no exponent), and its inverse
__device__ __forceinline__ float pow2_scale(float m, float& inv) {
  int e = (int)(__float_as_uint(m) >> 23);
  if (e < 1 || e > 253) e = 127;
  inv = __uint_as_float((uint32_t)e << 23);
  return __uint_as_float((uint32_t)(254 - e) << 23);
}

constexpr int kScWarps = 4;
constexpr int kScSteps = 4;                        // k32 steps loaded together

// One warp per 16 tokens.  NE: 8-expert tiles of the logits.  In a k32 step lane (g, c) (g = lane / 4,
// c = lane % 4) holds columns 8c .. 8c+7 of rows g and g + 8 of x and of row g of each 8 rows of Wg:
// the first four of them serve as k = 2c, 2c+1, 2c+8, 2c+9 of one k16 product, the others of a second.
template <int NE, bool F16>
__global__ void __launch_bounds__(kScWarps * 32) seq_scores_kernel(SeqBalArgs a) {
  using H = H16<F16>;
  constexpr int EP = NE * 8;
  __shared__ float dp_s[kScWarps][16][EP];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int D = a.D, E = a.E;
  const int rb = blockIdx.x * kScWarps + w;
  launch_dependents();
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  const int t0 = rb * 16 + g, t1 = t0 + 8;
  const bool v0 = t0 >= t_lo && t0 < t_hi, v1 = t1 >= t_lo && t1 < t_hi;
  const uint4* x0 = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + (size_t)t0 * D) + c;
  const uint4* x1 = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + (size_t)t1 * D) + c;
  const uint4* wr = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.wg) + (size_t)g * D) + c;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float acc[NE][2][4];
#pragma unroll
  for (int nt = 0; nt < NE; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[nt][h][q] = 0.f;
  const int steps = D / 32;
  if (__any_sync(0xffffffffu, v0 || v1)) {
    for (int s0 = 0; s0 < steps; s0 += kScSteps) {
      uint4 xa[kScSteps], xb[kScSteps];
#pragma unroll
      for (int u = 0; u < kScSteps; ++u) {
        const bool in = s0 + u < steps;
        xa[u] = in && v0 ? ld_stream(x0 + (s0 + u) * 4) : zero;
        xb[u] = in && v1 ? ld_stream(x1 + (s0 + u) * 4) : zero;
      }
#pragma unroll
      for (int u = 0; u < kScSteps; ++u) {
        if (s0 + u < steps) {
#pragma unroll
          for (int nt = 0; nt < NE; ++nt) {
            const uint4 b = nt * 8 + g < E ? __ldg(wr + (size_t)nt * D + (s0 + u) * 4) : zero;   // 8 rows on: D uint4s
            mma_16816<F16>(acc[nt][0], xa[u].x, xb[u].x, xa[u].y, xb[u].y, b.x, b.y);
            mma_16816<F16>(acc[nt][1], xa[u].z, xb[u].z, xa[u].w, xb[u].w, b.z, b.w);
          }
        }
      }
    }
  }
  // lane (g, c): logits of rows t0 and t1 (r = 0, 1), experts nt * 8 + 2c and + 1
  float l[2][NE][2];
#pragma unroll
  for (int nt = 0; nt < NE; ++nt)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int e = nt * 8 + 2 * c + q;
      const float b = e < E && a.bias ? a.bias[e] : 0.f;
#pragma unroll
      for (int r = 0; r < 2; ++r) l[r][nt][q] = e < E ? acc[nt][0][2 * r + q] + acc[nt][1][2 * r + q] + b : -INFINITY;
    }
#pragma unroll
  for (int r = 0; r < 2; ++r) {                    // softmax
    float m = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NE; ++nt) m = fmaxf(m, fmaxf(l[r][nt][0], l[r][nt][1]));
    m = quad_max(m);
    float z = 0.f;
#pragma unroll
    for (int nt = 0; nt < NE; ++nt)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        l[r][nt][q] = nt * 8 + 2 * c + q < E ? expf(l[r][nt][q] - m) : 0.f;
        z += l[r][nt][q];
      }
    const float iz = 1.0f / quad_sum(z);
#pragma unroll
    for (int nt = 0; nt < NE; ++nt)
#pragma unroll
      for (int q = 0; q < 2; ++q) l[r][nt][q] *= iz;
  }
  // the gates' gradients of the 16 tokens: scattered to their experts, each token by one lane
  if (a.dgate) {
    float* dp = &dp_s[w][0][0];
    for (int i = lane; i < 16 * EP; i += 32) dp[i] = 0.f;
    __syncwarp();
    const int t = rb * 16 + lane;
    if (lane < 16 && t >= t_lo && t < t_hi) {
      const int ns = slots_of(a, t);
      for (int k = 0; k < ns; ++k) {
        const int e = a.topk_idx[(size_t)t * a.Kmax + k];
        if (e >= 0 && e < E) dp[lane * EP + e] += a.dgate[(size_t)t * a.Kmax + k];
      }
    }
    __syncwarp();
  }
  grid_dependency_wait();                          // from here on: what count wrote
  const float aux = a.aux_scale / (float)max(*a.live, 1);
  float dl[2][NE][2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int t = r ? t1 : t0;
    const bool live = r ? v1 : v0;
    const int2 tk = live ? a.tok[t] : make_int2(-1, 0);
    const float coef = __int_as_float(tk.y);
    float dp[NE][2], share = 0.f, pc = 0.f;
#pragma unroll
    for (int nt = 0; nt < NE; ++nt)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int e = nt * 8 + 2 * c + q;
        const float C = tk.x >= 0 && e < E ? coef * (float)a.counts[(size_t)tk.x * E + e] : 0.f;
        share += l[r][nt][q] * C;
        dp[nt][q] = aux * C + (a.dgate ? dp_s[w][g + 8 * r][e] : 0.f);
        pc += l[r][nt][q] * dp[nt][q];
      }
    share = quad_sum(share);
    pc = quad_sum(pc);
    if (c == 0 && t < a.T) a.tok_loss[t] = tk.x >= 0 ? share : 0.f;
#pragma unroll
    for (int nt = 0; nt < NE; ++nt)
#pragma unroll
      for (int q = 0; q < 2; ++q) dl[r][nt][q] = tk.x >= 0 ? l[r][nt][q] * (dp[nt][q] - pc) : 0.f;
  }
  if (!a.grads || rb * 16 >= a.T) return;
  // db of the 16 tokens
#pragma unroll
  for (int nt = 0; nt < NE; ++nt)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float s = dl[0][nt][q] + dl[1][nt][q];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (g == 0) a.db_part[(size_t)rb * EP + nt * 8 + 2 * c + q] = s;
    }
  // fragments of dl and of its transpose
  float sr[2] = {1.f, 1.f}, sb = 1.f;
  if (F16) {
    float mr[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mr[r] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NE; ++nt) mr[r] = fmaxf(mr[r], fmaxf(fabsf(dl[r][nt][0]), fabsf(dl[r][nt][1])));
      mr[r] = quad_max(mr[r]);
      float inv;
      sr[r] = pow2_scale(mr[r], inv);
      if (c == 0) a.scales[(size_t)rb * kSbScales + g + 8 * r] = inv;
    }
    float mb = fmaxf(mr[0], mr[1]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    float inv;
    sb = pow2_scale(mb, inv);
    if (lane == 0) a.scales[(size_t)rb * kSbScales + 16] = inv;
  }
  uint32_t hi[2][NE], lo[2][NE], hit[2][NE], lot[2][NE];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int nt = 0; nt < NE; ++nt) {
      auto split = [](float u, float v, uint32_t& h, uint32_t& lw) {
        h = H::pack(u, v);
        const float2 f = H::unpack(h);
        lw = H::pack(u - f.x, v - f.y);
      };
      split(dl[r][nt][0] * sr[r], dl[r][nt][1] * sr[r], hi[r][nt], lo[r][nt]);
      if (F16) split(dl[r][nt][0] * sb, dl[r][nt][1] * sb, hit[r][nt], lot[r][nt]);
      else { hit[r][nt] = hi[r][nt]; lot[r][nt] = lo[r][nt]; }
      hit[r][nt] = movm_t(hit[r][nt]);
      lot[r][nt] = movm_t(lot[r][nt]);
    }
  constexpr int NF = NE == 1 ? 1 : NE;             // fragments (512 bytes) of each kind in a block
  uint4* fa = a.frag + (size_t)rb * 2 * NF * 32 + lane;
  uint4* ft = fa + NF * 32;
  if (NE == 1) {                                   // k = 0..7 the hi parts, 8..15 the lo parts
    fa[0] = make_uint4(hi[0][0], hi[1][0], lo[0][0], lo[1][0]);
    ft[0] = make_uint4(hit[0][0], lot[0][0], hit[1][0], lot[1][0]);
  } else {
#pragma unroll
    for (int p = 0; p < NE / 2; ++p) {             // 16 experts: hi, then lo
      fa[(2 * p) * 32] = make_uint4(hi[0][2 * p], hi[1][2 * p], hi[0][2 * p + (NE > 1)], hi[1][2 * p + (NE > 1)]);
      fa[(2 * p + 1) * 32] = make_uint4(lo[0][2 * p], lo[1][2 * p], lo[0][2 * p + (NE > 1)], lo[1][2 * p + (NE > 1)]);
      ft[(2 * p) * 32] = make_uint4(hit[0][2 * p], hit[0][2 * p + (NE > 1)], hit[1][2 * p], hit[1][2 * p + (NE > 1)]);
      ft[(2 * p + 1) * 32] = make_uint4(lot[0][2 * p], lot[0][2 * p + (NE > 1)], lot[1][2 * p], lot[1][2 * p + (NE > 1)]);
    }
  }
}

// ---------------------------------------------------------------- grads, 16-bit types
// One warp per (64 columns, range of 16-token blocks), dWg's slice in registers over the range.
//   dWg: product j takes column 8n + j as its n: lane (g, c) reads columns 8g .. 8g+7 of rows 2c, 2c+1,
//        2c+8, 2c+9, whole 128-byte lines.
//   dx:  of 32 columns at a time, product j takes column 8 (n / 2) + 2j + n % 2 as its n: lane (g, c)
//        then holds columns 8c .. 8c+7 of rows g and g + 8.
template <int NE, bool F16>
__global__ void __launch_bounds__(128) seq_grads_kernel(SeqBalArgs a) {
  using H = H16<F16>;
  constexpr int NF = NE == 1 ? 1 : NE;
  constexpr int NK = NE <= 2 ? 1 : NE / 2;         // 16-expert tiles
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int D = a.D, E = a.E;
  const int job = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int slabs = D / 64;
  launch_dependents();
  if (job >= slabs * a.ranges) return;
  const int range = job / slabs, col = (job % slabs) * 64;
  const int nblk = (a.T + 15) / 16;
  const int b0 = range * a.blocks_per_range, b1 = min(nblk, b0 + a.blocks_per_range);
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  // gate weight fragments of dx: rows e = 2c, 2c+1 (b0) and 2c+8, 2c+9 (b1) of 16 experts
  uint32_t wb[NK][8][NE == 1 ? 1 : 2];
  const uint16_t* wg = static_cast<const uint16_t*>(a.wg);
#pragma unroll
  for (int p = 0; p < NK; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int h = 0; h < (NE == 1 ? 1 : 2); ++h) {
        const int e = p * 16 + h * 8 + 2 * c, d = col + 32 * (j >> 2) + 8 * (g >> 1) + 2 * (j & 3) + (g & 1);
        const uint32_t u = e < E ? wg[(size_t)e * D + d] : 0u, v = e + 1 < E ? wg[(size_t)(e + 1) * D + d] : 0u;
        wb[p][j][h] = u | (v << 16);
      }
  float acc[NK][8][4];
#pragma unroll
  for (int p = 0; p < NK; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[p][j][q] = 0.f;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + col + 8 * g;
  auto load_x = [&](int b, uint4* r) {             // rows 2c, 2c+1, 2c+8, 2c+9 of block b
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = b * 16 + 2 * c + (i & 1) + 8 * (i >> 1);
      r[i] = t >= t_lo && t < t_hi ? ld_stream(x + (size_t)t * D) : zero;
    }
  };
  uint4 xn[4];
  if (b0 < b1) load_x(b0, xn);
  grid_dependency_wait();
  for (int b = b0; b < b1; ++b) {
    uint4 xr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xr[i] = xn[i];
    const int t0 = b * 16 + g, t1 = t0 + 8;
    const bool v0 = t0 >= t_lo && t0 < t_hi, v1 = t1 >= t_lo && t1 < t_hi;
    uint16_t* d0 = static_cast<uint16_t*>(a.dx) + (size_t)t0 * D + col + 8 * c;
    uint16_t* d1 = d0 + (size_t)8 * D;
    uint4 old[2][2];
    if (a.dx && a.accumulate) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        old[h][0] = v0 ? __ldcs(reinterpret_cast<const uint4*>(d0 + 32 * h)) : zero;
        old[h][1] = v1 ? __ldcs(reinterpret_cast<const uint4*>(d1 + 32 * h)) : zero;
      }
    }
    const uint4* fa = a.frag + (size_t)b * 2 * NF * 32 + lane;
    uint4 A[NF], At[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      A[f] = fa[f * 32];
      At[f] = fa[(NF + f) * 32];
    }
    float inv0 = 1.f, inv1 = 1.f, invb = 1.f;
    if (F16) {
      const float* sc = a.scales + (size_t)b * kSbScales;
      inv0 = sc[g]; inv1 = sc[g + 8]; invb = sc[16];
    }
    if (b + 1 < b1) load_x(b + 1, xn);
    // ---- dWg += dl^T x
    const uint32_t* xw[4] = {reinterpret_cast<const uint32_t*>(&xr[0]), reinterpret_cast<const uint32_t*>(&xr[1]),
                             reinterpret_cast<const uint32_t*>(&xr[2]), reinterpret_cast<const uint32_t*>(&xr[3])};
#pragma unroll
    for (int j = 0; j < 8; ++j) {                  // columns 8g + j: (row, next row) pairs
      const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
      const uint32_t p0 = __byte_perm(xw[0][j >> 1], xw[1][j >> 1], sel);
      const uint32_t p1 = __byte_perm(xw[2][j >> 1], xw[3][j >> 1], sel);
#pragma unroll
      for (int p = 0; p < NK; ++p) {
        if (F16) {                                 // the block's scale is taken out of each block's product
          float d4[4] = {0.f, 0.f, 0.f, 0.f};
          mma_16816<F16>(d4, At[NE == 1 ? 0 : 2 * p].x, At[NE == 1 ? 0 : 2 * p].y, At[NE == 1 ? 0 : 2 * p].z,
                         At[NE == 1 ? 0 : 2 * p].w, p0, p1);
          if (NE > 1) mma_16816<F16>(d4, At[(2 * p + 1) % NF].x, At[(2 * p + 1) % NF].y, At[(2 * p + 1) % NF].z, At[(2 * p + 1) % NF].w, p0, p1);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[p][j][q] = fmaf(d4[q], invb, acc[p][j][q]);
        } else {
          mma_16816<F16>(acc[p][j], At[NE == 1 ? 0 : 2 * p].x, At[NE == 1 ? 0 : 2 * p].y, At[NE == 1 ? 0 : 2 * p].z,
                         At[NE == 1 ? 0 : 2 * p].w, p0, p1);
          if (NE > 1) mma_16816<F16>(acc[p][j], At[(2 * p + 1) % NF].x, At[(2 * p + 1) % NF].y, At[(2 * p + 1) % NF].z, At[(2 * p + 1) % NF].w, p0, p1);
        }
      }
    }
    // ---- dx = dl Wg
    if (a.dx) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float o0[8], o1[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float d4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int p = 0; p < NK; ++p) {
            const uint32_t w0 = wb[p][4 * h + j][0], w1 = wb[p][4 * h + j][NE == 1 ? 0 : 1];
            const uint4 ah = A[NE == 1 ? 0 : 2 * p];
            mma_16816<F16>(d4, ah.x, ah.y, ah.z, ah.w, w0, w1);
            if (NE > 1) {
              const uint4 al = A[(2 * p + 1) % NF];
              mma_16816<F16>(d4, al.x, al.y, al.z, al.w, w0, w1);
            }
          }
          o0[2 * j] = d4[0]; o0[2 * j + 1] = d4[1]; o1[2 * j] = d4[2]; o1[2 * j + 1] = d4[3];
        }
        uint32_t r0[4], r1[4];
        const uint32_t* q0 = reinterpret_cast<const uint32_t*>(&old[h][0]);
        const uint32_t* q1 = reinterpret_cast<const uint32_t*>(&old[h][1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 f0 = make_float2(0.f, 0.f), f1 = f0;
          if (a.accumulate) {
            f0 = H::unpack(q0[i]);
            f1 = H::unpack(q1[i]);
          }
          r0[i] = H::pack(fmaf(o0[2 * i], inv0, f0.x), fmaf(o0[2 * i + 1], inv0, f0.y));
          r1[i] = H::pack(fmaf(o1[2 * i], inv1, f1.x), fmaf(o1[2 * i + 1], inv1, f1.y));
        }
        if (v0) __stcs(reinterpret_cast<uint4*>(d0 + 32 * h), make_uint4(r0[0], r0[1], r0[2], r0[3]));
        if (v1) __stcs(reinterpret_cast<uint4*>(d1 + 32 * h), make_uint4(r1[0], r1[1], r1[2], r1[3]));
      }
    }
  }
  // this range's partial dWg: expert row g (and g + 8), columns 16c .. 16c+15
  float* part = a.partials + (size_t)range * E * D + col + 16 * c;
#pragma unroll
  for (int p = 0; p < NK; ++p) {
#pragma unroll
    for (int r = 0; r < (NE == 1 ? 1 : 2); ++r) {
      const int e = p * 16 + r * 8 + g;
      if (e < E) {
#pragma unroll
        for (int s = 0; s < 2; ++s)                // columns 16c + 8s + j
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            float f[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              f[q] = NE == 1 ? acc[p][4 * v + q][s] + acc[p][4 * v + q][2 + s] : acc[p][4 * v + q][2 * r + s];
            *reinterpret_cast<float4*>(part + (size_t)e * D + 8 * s + 4 * v) = make_float4(f[0], f[1], f[2], f[3]);
          }
      }
    }
  }
}

// ---------------------------------------------------------------- fp32
// FFMA throughout (a tensor core would round x).  One warp per four tokens: lane l holds columns
// 4l + 128 i of their rows and of Wg's.
constexpr int kF32Tok = 4;

template <int EP>
__global__ void __launch_bounds__(128) seq_scores_f32_kernel(SeqBalArgs a) {
  __shared__ float db_s[4][EP];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int D = a.D, E = a.E;
  const int tb = blockIdx.x * 16 + w * kF32Tok;
  launch_dependents();
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  float l[kF32Tok][EP];
#pragma unroll
  for (int i = 0; i < kF32Tok; ++i)
#pragma unroll
    for (int e = 0; e < EP; ++e) l[i][e] = 0.f;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* x = static_cast<const float*>(a.x);
  const float* wg = static_cast<const float*>(a.wg);
  for (int d = lane * 4; d < D; d += 128) {
    float4 xv[kF32Tok];
#pragma unroll
    for (int i = 0; i < kF32Tok; ++i) {
      const int t = tb + i;
      xv[i] = t >= t_lo && t < t_hi ? __ldg(reinterpret_cast<const float4*>(x + (size_t)t * D + d)) : zero;
    }
#pragma unroll
    for (int e = 0; e < EP; ++e) {
      if (e < E) {
        const float4 wv = __ldg(reinterpret_cast<const float4*>(wg + (size_t)e * D + d));
#pragma unroll
        for (int i = 0; i < kF32Tok; ++i)
          l[i][e] = fmaf(xv[i].x, wv.x, fmaf(xv[i].y, wv.y, fmaf(xv[i].z, wv.z, fmaf(xv[i].w, wv.w, l[i][e]))));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kF32Tok; ++i)
#pragma unroll
    for (int e = 0; e < EP; ++e)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], o);
  // every lane holds every sum; lane e keeps expert e's
  float db = 0.f;
  grid_dependency_wait();
  const float aux = a.aux_scale / (float)max(*a.live, 1);
#pragma unroll
  for (int i = 0; i < kF32Tok; ++i) {
    const int t = tb + i;
    float mine = -INFINITY;
#pragma unroll
    for (int e = 0; e < EP; ++e)
      if (lane == e && e < E) mine = l[i][e] + (a.bias ? a.bias[e] : 0.f);
    const int2 tk = t >= t_lo && t < t_hi ? a.tok[t] : make_int2(-1, 0);
    float m = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float pe = lane < E ? expf(mine - m) : 0.f;
    float z = pe;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float P = pe * (1.0f / z);
    const float C = tk.x >= 0 && lane < E ? __int_as_float(tk.y) * (float)a.counts[(size_t)tk.x * E + lane] : 0.f;
    float dp = aux * C;
    if (a.dgate && tk.x >= 0) {
      const int ns = slots_of(a, t);
      for (int k = 0; k < ns; ++k)
        if (a.topk_idx[(size_t)t * a.Kmax + k] == lane) dp += a.dgate[(size_t)t * a.Kmax + k];
    }
    float share = P * C, pc = P * dp;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      share += __shfl_xor_sync(0xffffffffu, share, o);
      pc += __shfl_xor_sync(0xffffffffu, pc, o);
    }
    const float dl = tk.x >= 0 && lane < E ? P * (dp - pc) : 0.f;
    db += dl;
    if (t < a.T) {
      if (lane == 0) a.tok_loss[t] = tk.x >= 0 ? share : 0.f;
      if (a.grads && lane < EP) a.dl[(size_t)t * EP + lane] = dl;
    }
  }
  if (!a.grads) return;
  if (lane < EP) db_s[w][lane] = db;
  __syncthreads();
  if (threadIdx.x < EP)
    a.db_part[(size_t)blockIdx.x * EP + threadIdx.x] =
        (db_s[0][threadIdx.x] + db_s[1][threadIdx.x]) + (db_s[2][threadIdx.x] + db_s[3][threadIdx.x]);
}

// One warp per (128 columns, range of 16-token blocks): lane l owns four columns, its slice of dWg in
// registers over the range.  D is a multiple of 64: the upper half warp of a last half slab idles.
template <int EP>
__global__ void __launch_bounds__(128) seq_grads_f32_kernel(SeqBalArgs a) {
  const int lane = threadIdx.x & 31;
  const int D = a.D, E = a.E;
  const int job = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int slabs = (D + 127) / 128;
  launch_dependents();
  if (job >= slabs * a.ranges) return;
  const int range = job / slabs, col = (job % slabs) * 128 + lane * 4;
  const int t_begin = range * a.blocks_per_range * 16, t_end = min(a.T, t_begin + a.blocks_per_range * 16);
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  float4 acc[EP];
#pragma unroll
  for (int e = 0; e < EP; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  grid_dependency_wait();
  if (col >= D) return;
  const float* x = static_cast<const float*>(a.x) + col;
  const float* wg = static_cast<const float*>(a.wg) + col;
  float* dx = a.dx ? static_cast<float*>(a.dx) + col : nullptr;
#pragma unroll 2
  for (int t = max(t_begin, t_lo); t < min(t_end, t_hi); ++t) {
    const float4 xv = __ldg(reinterpret_cast<const float4*>(x + (size_t)t * D));
    const float* dr = a.dl + (size_t)t * EP;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (dx && a.accumulate) o = *reinterpret_cast<const float4*>(dx + (size_t)t * D);
#pragma unroll
    for (int e = 0; e < EP; ++e) {
      if (e < E) {
        const float d = dr[e];
        acc[e].x = fmaf(d, xv.x, acc[e].x); acc[e].y = fmaf(d, xv.y, acc[e].y);
        acc[e].z = fmaf(d, xv.z, acc[e].z); acc[e].w = fmaf(d, xv.w, acc[e].w);
        if (dx) {
          const float4 wv = __ldg(reinterpret_cast<const float4*>(wg + (size_t)e * D));
          o.x = fmaf(d, wv.x, o.x); o.y = fmaf(d, wv.y, o.y); o.z = fmaf(d, wv.z, o.z); o.w = fmaf(d, wv.w, o.w);
        }
      }
    }
    if (dx) *reinterpret_cast<float4*>(dx + (size_t)t * D) = o;
  }
  float* part = a.partials + (size_t)range * E * D + col;
#pragma unroll
  for (int e = 0; e < EP; ++e)
    if (e < E) *reinterpret_cast<float4*>(part + (size_t)e * D) = acc[e];
}

// ---------------------------------------------------------------- finish
__device__ __forceinline__ double block_sum_f64(double v, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kFinThreads / 32; ++w) s += sh[w];
  return s;
}

// Blocks by role, all sums in a fixed order: 32 elements of dWg each (8 warps over the ranges); one for
// each expert's db; one for each sequence's loss; one for the mean loss.
__global__ void __launch_bounds__(kFinThreads) seq_finish_kernel(SeqBalArgs a, int ep, int wg_blocks, int db_blocks) {
  __shared__ double sh[kFinThreads / 32];
  __shared__ float ws[kFinThreads / 32][32];
  constexpr int NW = kFinThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int blk = blockIdx.x;
  grid_dependency_wait();
  if (blk < wg_blocks) {
    const int i = blk * 32 + lane;                 // E * D is a multiple of 64
    const size_t stride = (size_t)a.E * a.D;
    float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = w; k < a.ranges; k += NW * 8)
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (k + u * NW < a.ranges) r[u] += __ldcg(a.partials + (size_t)(k + u * NW) * stride + i);
    ws[w][lane] = ((r[0] + r[1]) + (r[2] + r[3])) + ((r[4] + r[5]) + (r[6] + r[7]));
    __syncthreads();
    if (w == 0) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) t += ws[k][lane];
      a.dwg[i] = t;
    }
    return;
  }
  blk -= wg_blocks;
  if (blk < db_blocks) {
    const int nblk = (a.T + 15) / 16;
    double s = 0.0;
    for (int k = tid; k < nblk; k += kFinThreads) s += (double)__ldcg(a.db_part + (size_t)k * ep + blk);
    s = block_sum_f64(s, sh);
    if (tid == 0) a.dbias[blk] = (float)s;
    return;
  }
  blk -= db_blocks;
  int lo, hi;
  if (blk < a.n_seqs) {
    lo = a.offsets ? min(max(a.offsets[blk], 0), a.T) : blk * a.seq_len;
    hi = a.offsets ? min(max(a.offsets[blk + 1], lo), a.T) : lo + a.seq_len;
  } else {
    live_rows(a, lo, hi);
  }
  double s = 0.0;
  for (int t = lo + tid; t < hi; t += kFinThreads) s += (double)__ldcg(a.tok_loss + t);
  s = block_sum_f64(s, sh);
  if (tid == 0) {
    if (blk < a.n_seqs) a.seq_loss[blk] = (float)s;
    else *a.loss = (float)(s / (double)max(*a.live, 1));
  }
}

template <typename... P, typename... Q>
cudaError_t chained(void (*k)(P...), int grid, int threads, cudaStream_t s, Q... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

template <int NE, bool F16>
cudaError_t launch16(const SeqBalArgs& a, cudaStream_t s) {
  const int nblk = (a.T + 15) / 16;
  cudaError_t e = chained(seq_scores_kernel<NE, F16>, (nblk + kScWarps - 1) / kScWarps, kScWarps * 32, s, a);
  if (e != cudaSuccess || !a.grads) return e;
  return chained(seq_grads_kernel<NE, F16>, (a.D / 64 * a.ranges + 3) / 4, 128, s, a);
}
template <int EP>
cudaError_t launch32(const SeqBalArgs& a, cudaStream_t s) {
  cudaError_t e = chained(seq_scores_f32_kernel<EP>, (a.T + 15) / 16, 128, s, a);
  if (e != cudaSuccess || !a.grads) return e;
  return chained(seq_grads_f32_kernel<EP>, ((a.D + 127) / 128 * a.ranges + 3) / 4, 128, s, a);
}
template <bool F16>
cudaError_t launch16_e(const SeqBalArgs& a, cudaStream_t s) {
  return a.E <= 8 ? launch16<1, F16>(a, s) : a.E <= 16 ? launch16<2, F16>(a, s) : launch16<4, F16>(a, s);
}

}  // namespace

int seq_balance_ep(int E) { return E <= 8 ? 8 : E <= 16 ? 16 : 32; }

void seq_balance_plan(int T, int D, int dtype, int* ranges, int* blocks_per_range) {
  const int slabs = dtype == MOE_F32 ? (D + 127) / 128 : D / 64;
  const int nblk = (T + 15) / 16;
  int r = kSbJobs / slabs;
  if (r > nblk) r = nblk;
  if (r < 1) r = 1;
  *blocks_per_range = (nblk + r - 1) / r;
  *ranges = *blocks_per_range > 0 ? (nblk + *blocks_per_range - 1) / *blocks_per_range : 0;
}

cudaError_t launch_seq_balance(const SeqBalArgs& a, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(a.counts, 0, (size_t)a.n_seqs * a.E * sizeof(int32_t), s);
  if (e == cudaSuccess) e = cudaMemsetAsync(a.live, 0, sizeof(int), s);
  if (e != cudaSuccess) return e;
  seq_count_kernel<<<(a.T + kCountThreads - 1) / kCountThreads, kCountThreads, 0, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.dtype == MOE_F32)
    e = a.E <= 8 ? launch32<8>(a, s) : a.E <= 16 ? launch32<16>(a, s) : launch32<32>(a, s);
  else
    e = a.dtype == MOE_F16 ? launch16_e<true>(a, s) : launch16_e<false>(a, s);
  if (e != cudaSuccess) return e;
  const int wg_blocks = a.dwg ? a.E * a.D / 32 : 0, db_blocks = a.dbias ? a.E : 0;
  return chained(seq_finish_kernel, wg_blocks + db_blocks + a.n_seqs + 1, kFinThreads, s, a, seq_balance_ep(a.E), wg_blocks,
                 db_blocks);
}

}  // namespace moe
