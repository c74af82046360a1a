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
// is a by-product of the softmax's backward.  Rows of no sequence take no part, whatever their
// x holds, and their dx stays.
//
// Four launches, each bound by memory, none with a barrier in its loop:
//   count   sequence and factor of every token, counts (integer atomics)
//   scores  logits, softmax, dl: reads x once
//   grads   dx and the partial sums of dWg: reads x again (from L2 where it fits), dx in and out
//   finish  the partial sums of dWg and db in a fixed order, the losses
// They are chained by programmatic dependent launch: scores forms its logits while count runs.
//
// The 16-bit kernels' mma.sync fragments are 16 consecutive bytes of a row in every lane.  Where an
// index is summed over (the columns in the logits) or names an output (the columns of dx and of
// dWg) the order in which a fragment holds it is free, so each lane copies the pieces of rows that
// will be its own fragments and reads back only what it copied: a ring of cp.async stages that needs
// no barrier, no swizzle and no ldmatrix, and keeps kilobytes of each warp in flight.  dWg sums over
// tokens, whose pairs lie in different rows: two rows' pieces are interleaved in registers.
// dl goes between the kernels already in fragment order, as it is and transposed (movmatrix), in
// 16-bit parts that add up to it: for dx two; for dWg, which stays in fp32, three of bf16 (24 bits)
// or two of fp16 (22 bits below the largest of its 16 tokens; each row of dx has a scale of its own).
// With E <= 8 two parts share one k16 step.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kCountThreads = 256;
constexpr int kOffSmem = 2048;                     // offsets kept in shared memory up to this many
constexpr int kCountSmall = 4096;                  // tokens, and counts, that one block takes alone
constexpr int kFinThreads = 256;

// 16 bytes into this lane's own slot (zeros where !in): read back by the lane alone, after cp_wait
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
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
// (sequence, expert) keys of a warp merged first, as in the frequency kernel).  SMALL: one block, the
// counts in shared memory.  T = 512: 1.9 us less than clearing and adding to them in global memory.
template <bool SMALL>
__global__ void __launch_bounds__(SMALL ? 1024 : kCountThreads) seq_count_kernel(SeqBalArgs a) {
  __shared__ int off_s[kOffSmem];
  __shared__ int hist[SMALL ? kCountSmall : 1];
  __shared__ int full_s;
  launch_dependents();
  const int tid = threadIdx.x, n = a.n_seqs, nt = blockDim.x;
  const int* off = a.offsets;
  const bool in_smem = n + 1 <= kOffSmem;
  if (SMALL)
    for (int i = tid; i < n * a.E; i += nt) hist[i] = 0;
  if (tid == 0) full_s = 0;
  if (off && in_smem) {
    for (int i = tid; i <= n; i += nt) off_s[i] = off[i];
    off = off_s;
  }
  __syncthreads();
  // sequences that hold a row: by the first block where it has the offsets at hand, else by all blocks
  if (off && (!in_smem || blockIdx.x == 0)) {
    int full = 0;
    for (int b = (in_smem ? 0 : blockIdx.x * nt) + tid; b < n; b += in_smem ? nt : gridDim.x * nt) {
      const int lo = off[b], hi = off[b + 1];
      if (lo < 0 || hi < lo || hi > a.T) set_status(a.status, DEV_BAD_INDEX, 410);
      full += hi > lo;
    }
    full = __reduce_add_sync(0xffffffffu, full);
    if ((tid & 31) == 0 && full) atomicAdd(in_smem ? &full_s : a.live, full);
  }
  for (int t0 = blockIdx.x * nt; t0 < a.T; t0 += gridDim.x * nt) {
    const int t = t0 + tid;
    int sid = -1, len = 0;
    if (t < a.T) {
      if (off) {
        int lo = 0, hi = n;                        // the last sequence that starts at or before t
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
      if (SMALL) {
        if (key >= 0) atomicAdd(&hist[key], 1);
      } else {
        const unsigned same = __match_any_sync(0xffffffffu, key);
        if (key >= 0 && (tid & 31) == __ffs(same) - 1) atomicAdd(&a.counts[key], __popc(same));
      }
    }
  }
  __syncthreads();
  if (SMALL)
    for (int i = tid; i < n * a.E; i += nt) a.counts[i] = hist[i];
  if (blockIdx.x == 0 && tid == 0 && (in_smem || !a.offsets)) *a.live = a.offsets ? full_s : n;
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
constexpr int kScRing = 12;                        // k32 steps in flight: 12 KB a warp, 16 warps an SM
constexpr int kScSmem = kScWarps * kScRing * 1024;
constexpr int kGateAhead = 4;                      // slots of a token whose gate gradients are loaded ahead

// Parts of dl that dx and dWg take, and so the 512-byte fragments of a 16-token block, by experts
// (NE tiles of 8) and type.
template <int NE, bool F16> struct Parts {
  static constexpr int NK = NE <= 2 ? 1 : NE / 2;           // 16-expert tiles
  static constexpr int A = NE == 1 ? 1 : 2 * NK;            // for dx
  static constexpr int T = F16 ? A : NE == 1 ? 2 : 3 * NK;  // for dWg
};

// One warp per 16 tokens.  NE: 8-expert tiles of the logits.  In a k32 step lane (g, c) (g = lane / 4,
// c = lane % 4) holds columns 8c .. 8c+7 of rows g and g + 8 of x and of row g of each 8 rows of Wg:
// the first four of them serve as k = 2c, 2c+1, 2c+8, 2c+9 of one k16 product, the others of a second.
template <int NE, bool F16>
__global__ void __launch_bounds__(kScWarps * 32) seq_scores_kernel(SeqBalArgs a) {
  using H = H16<F16>;
  constexpr int EP = NE * 8;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float dp_s[kScWarps][16][EP];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int D = a.D, E = a.E;
  const int rb = blockIdx.x * kScWarps + w;
  launch_dependents();
  const int t0 = rb * 16 + g, t1 = t0 + 8;
  const bool in0 = t0 < a.T, in1 = t1 < a.T;
  const uint16_t* x0 = static_cast<const uint16_t*>(a.x) + (in0 ? (size_t)t0 * D : 0) + 8 * c;
  const uint16_t* x1 = static_cast<const uint16_t*>(a.x) + (in1 ? (size_t)t1 * D : 0) + 8 * c;
  const uint4* wr = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.wg) + (size_t)g * D) + c;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint8_t* mine = ring + (size_t)w * kScRing * 1024 + lane * 16;
  const uint32_t dst = smem_u32(mine);
  const int steps = D / 32;
#pragma unroll
  for (int s = 0; s < kScRing; ++s) {
    if (s < steps) {
      cp16(dst + s * 1024, x0 + s * 32, in0);
      cp16(dst + s * 1024 + 512, x1 + s * 32, in1);
    }
    cp_commit();
  }
  // what the rest needs of the token of this lane (lanes 0..15), on its way meanwhile
  const int tl = rb * 16 + lane;
  const bool gated = a.dgate && lane < 16 && tl < a.T;
  const int ns = gated ? slots_of(a, tl) : 0;
  int ge[kGateAhead];
  float gv[kGateAhead];
#pragma unroll
  for (int k = 0; k < kGateAhead; ++k) {
    ge[k] = gated && k < a.Kmax ? a.topk_idx[(size_t)tl * a.Kmax + k] : -1;
    gv[k] = gated && k < a.Kmax ? a.dgate[(size_t)tl * a.Kmax + k] : 0.f;
  }
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  const bool v0 = t0 >= t_lo && t0 < t_hi, v1 = t1 >= t_lo && t1 < t_hi;
  float acc[NE][2][4];
#pragma unroll
  for (int nt = 0; nt < NE; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[nt][h][q] = 0.f;
  int slot = 0;
#pragma unroll 4
  for (int s = 0; s < steps; ++s) {
    uint4 b[NE];
#pragma unroll
    for (int nt = 0; nt < NE; ++nt) b[nt] = nt * 8 + g < E ? __ldg(wr + (size_t)nt * D + s * 4) : zero;   // 8 rows on: D uint4s
    cp_wait<kScRing - 1>();
    const uint4 xa = *reinterpret_cast<const uint4*>(mine + slot * 1024);
    const uint4 xb = *reinterpret_cast<const uint4*>(mine + slot * 1024 + 512);
#pragma unroll
    for (int nt = 0; nt < NE; ++nt) {
      mma_16816<F16>(acc[nt][0], xa.x, xb.x, xa.y, xb.y, b[nt].x, b[nt].y);
      mma_16816<F16>(acc[nt][1], xa.z, xb.z, xa.w, xb.w, b[nt].z, b[nt].w);
    }
    if (s + kScRing < steps) {                     // the slot's contents are in registers: refill it
      cp16(dst + slot * 1024, x0 + (s + kScRing) * 32, in0);
      cp16(dst + slot * 1024 + 512, x1 + (s + kScRing) * 32, in1);
    }
    cp_commit();
    slot = slot + 1 == kScRing ? 0 : slot + 1;
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
    if (tl >= t_lo && tl < t_hi) {                 // ns = 0 on the other lanes
#pragma unroll
      for (int k = 0; k < kGateAhead; ++k)
        if (k < ns && ge[k] >= 0 && ge[k] < E) dp[lane * EP + ge[k]] += gv[k];
      for (int k = kGateAhead; k < ns; ++k) {
        const int e = a.topk_idx[(size_t)tl * a.Kmax + k];
        if (e >= 0 && e < E) dp[lane * EP + e] += a.dgate[(size_t)tl * a.Kmax + k];
      }
    }
    __syncwarp();
  }
  grid_dependency_wait();                          // from here on: what count wrote
  const float aux = a.aux_scale / (float)max(*a.live, 1);
  float dl[2][NE][2], loss16 = 0.f;
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
    share = tk.x >= 0 ? share : 0.f;
    if (c == 0 && t < a.T) a.tok_loss[t] = share;
    loss16 += share;
#pragma unroll
    for (int nt = 0; nt < NE; ++nt)
#pragma unroll
      for (int q = 0; q < 2; ++q) dl[r][nt][q] = tk.x >= 0 ? l[r][nt][q] * (dp[nt][q] - pc) : 0.f;
  }
  if (rb * 16 >= a.T) return;
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) loss16 += __shfl_xor_sync(0xffffffffu, loss16, o);
  if (lane == 0) a.blk_loss[rb] = loss16;
  if (!a.grads) return;
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
    float mr[2], inv[2], invb;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mr[r] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NE; ++nt) mr[r] = fmaxf(mr[r], fmaxf(fabsf(dl[r][nt][0]), fabsf(dl[r][nt][1])));
      mr[r] = quad_max(mr[r]);
      sr[r] = pow2_scale(mr[r], inv[r]);
    }
    float mb = fmaxf(mr[0], mr[1]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    sb = pow2_scale(mb, invb);
    if (c == 0) a.scales[(size_t)rb * 8 + g] = make_float4(inv[0], inv[1], invb, 0.f);
  }
  using P = Parts<NE, F16>;
  constexpr int NP = F16 ? 2 : 3;                  // parts
  uint32_t f[2][NP][NE], ft[2][NP][NE];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int nt = 0; nt < NE; ++nt) {
      auto split = [](float u, float v, uint32_t* part, int stride) {   // each part what the ones before leave
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          part[i * stride] = H::pack(u, v);
          const float2 h = H::unpack(part[i * stride]);
          u -= h.x;
          v -= h.y;
        }
      };
      split(dl[r][nt][0] * sr[r], dl[r][nt][1] * sr[r], &f[r][0][nt], NE);
      if (F16) split(dl[r][nt][0] * sb, dl[r][nt][1] * sb, &ft[r][0][nt], NE);
#pragma unroll
      for (int i = 0; i < NP; ++i) ft[r][i][nt] = movm_t(F16 ? ft[r][i][nt] : f[r][i][nt]);
    }
  uint4* fa = a.frag + (size_t)rb * (P::A + P::T) * 32 + lane;
  uint4* fw = fa + P::A * 32;
  if (NE == 1) {                                   // k (or m) = 0..7 the first part, 8..15 the second; then the third
    fa[0] = make_uint4(f[0][0][0], f[1][0][0], f[0][1][0], f[1][1][0]);
    fw[0] = make_uint4(ft[0][0][0], ft[0][1][0], ft[1][0][0], ft[1][1][0]);
    if (NP == 3) fw[32] = make_uint4(ft[0][NP - 1][0], 0u, ft[1][NP - 1][0], 0u);
  } else {
#pragma unroll
    for (int p = 0; p < P::NK; ++p)
#pragma unroll
      for (int i = 0; i < NP; ++i) {               // 16 experts: part after part
        constexpr int o = NE > 1;
        if (i < 2) fa[(2 * p + i) * 32] = make_uint4(f[0][i][2 * p], f[1][i][2 * p], f[0][i][2 * p + o], f[1][i][2 * p + o]);
        fw[(NP * p + i) * 32] = make_uint4(ft[0][i][2 * p], ft[0][i][2 * p + o], ft[1][i][2 * p], ft[1][i][2 * p + o]);
      }
  }
}

// ---------------------------------------------------------------- grads, 16-bit types
// One block per (64 columns, four ranges of 16-token blocks), a warp to a range, dWg's slice in
// registers over it; the four are added at the end.
//   dWg: product j takes column 8n + j as its n: lane (g, c) copies columns 8g .. 8g+7 of rows 2c, 2c+1,
//        2c+8, 2c+9, whole 128-byte lines.
//   dx:  of 32 columns at a time, product j takes column 8 (n / 2) + 2j + n % 2 as its n: lane (g, c)
//        then holds columns 8c .. 8c+7 of rows g and g + 8, and copies them of what is in dx.
template <int NE, bool F16> struct GradRing {
  using P = Parts<NE, F16>;
  static constexpr int Slots = 8 + P::A + P::T + (F16 ? 1 : 0);   // 512 bytes each: x 4, dx 4, dl, scales
  static constexpr int Stages = NE == 1 ? 3 : 2;                  // NE = 1: 17 KB a warp, 12 warps an SM
  static constexpr int Ring = 4 * Stages * Slots * 512;
  static constexpr int Sum = 4 * NE * 8 * 64 * 4;
  static constexpr int Smem = Ring > Sum ? Ring : Sum;
};
template <int NE, bool F16>
__global__ void __launch_bounds__(128, NE == 4 ? 2 : 3) seq_grads_kernel(SeqBalArgs a) {
  using H = H16<F16>;
  using P = Parts<NE, F16>;
  using R = GradRing<NE, F16>;
  constexpr int NK = P::NK, S = R::Stages, EP = NE * 8;
  extern __shared__ __align__(16) uint8_t ring[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int D = a.D, E = a.E;
  const int slabs = D / 64, group = blockIdx.x / slabs, col = (blockIdx.x % slabs) * 64;
  launch_dependents();
  const int nblk = (a.T + 15) / 16;
  const int b0 = (group * 4 + w) * a.blocks_per_range, b1 = min(nblk, b0 + a.blocks_per_range);
  const bool add = a.dx && a.accumulate;
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  uint8_t* mine = ring + (size_t)w * S * R::Slots * 512 + lane * 16;
  const uint32_t dst0 = smem_u32(mine);
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + col + 8 * g;
  uint16_t* dx = static_cast<uint16_t*>(a.dx) + col + 8 * c;
  auto copy_rows = [&](int b, int st) {            // x and dx of block b
    const uint32_t dst = dst0 + st * (R::Slots * 512);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = b * 16 + 2 * c + (i & 1) + 8 * (i >> 1);
      const bool in = t >= t_lo && t < t_hi;
      cp16(dst + i * 512, x + (in ? (size_t)t * D : 0), in);
    }
    if (add) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = b * 16 + g + 8 * (i & 1);
        const bool in = t >= t_lo && t < t_hi;
        cp16(dst + (4 + i) * 512, dx + (in ? (size_t)t * D : 0) + 32 * (i >> 1), in);
      }
    }
  };
  auto copy_parts = [&](int b, int st) {           // dl of block b
    const uint32_t dst = dst0 + st * (R::Slots * 512) + 8 * 512;
    const uint4* fr = a.frag + (size_t)b * (P::A + P::T) * 32 + lane;
#pragma unroll
    for (int i = 0; i < P::A + P::T; ++i) cp16(dst + i * 512, fr + i * 32, true);
    if (F16) cp16(dst + (P::A + P::T) * 512, a.scales + (size_t)b * 8 + g, true);
  };
#pragma unroll
  for (int st = 0; st < S; ++st)
    if (b0 + st < b1) copy_rows(b0 + st, st);
  // gate weight fragments of dx: rows e = 2c, 2c+1 (h = 0) and 2c+8, 2c+9 (h = 1) of 16 experts
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
  grid_dependency_wait();
#pragma unroll
  for (int st = 0; st < S; ++st) {
    if (b0 + st < b1) copy_parts(b0 + st, st);
    cp_commit();
  }
  int st = 0;
  for (int b = b0; b < b1; ++b) {
    cp_wait<S - 1>();
    const uint8_t* in = mine + st * (R::Slots * 512);
    auto slot = [&](int i) { return *reinterpret_cast<const uint4*>(in + i * 512); };
    uint4 xr[4], A[P::A], old[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xr[i] = slot(i);
#pragma unroll
    for (int i = 0; i < P::A; ++i) A[i] = slot(8 + i);
    float4 inv = make_float4(1.f, 1.f, 1.f, 0.f);
    if (F16) inv = *reinterpret_cast<const float4*>(in + (8 + P::A + P::T) * 512);
    // ---- dWg += dl^T x
    const uint32_t* xw[4] = {reinterpret_cast<const uint32_t*>(&xr[0]), reinterpret_cast<const uint32_t*>(&xr[1]),
                             reinterpret_cast<const uint32_t*>(&xr[2]), reinterpret_cast<const uint32_t*>(&xr[3])};
    constexpr int TP = P::T / NK;                  // fragments of a 16-expert tile
#pragma unroll
    for (int p = 0; p < NK; ++p) {
      uint4 At[TP];
#pragma unroll
      for (int i = 0; i < TP; ++i) At[i] = slot(8 + P::A + p * TP + i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {                // columns 8g + j: (row, next row) pairs
        const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
        const uint32_t p0 = __byte_perm(xw[0][j >> 1], xw[1][j >> 1], sel);
        const uint32_t p1 = __byte_perm(xw[2][j >> 1], xw[3][j >> 1], sel);
        // the block's product on its own, smallest part first, then one rounded addition (with fp16's scale)
        float d4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = TP - 1; i >= 0; --i) mma_16816<F16>(d4, At[i].x, At[i].y, At[i].z, At[i].w, p0, p1);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[p][j][q] = F16 ? fmaf(d4[q], inv.z, acc[p][j][q]) : acc[p][j][q] + d4[q];
      }
    }
    // ---- dx (+)= dl Wg
    if (add) {
#pragma unroll
      for (int i = 0; i < 4; ++i) old[i] = slot(4 + i);
    }
    if (a.dx) {
      const int t0 = b * 16 + g, t1 = t0 + 8;
      const bool v0 = t0 >= t_lo && t0 < t_hi, v1 = t1 >= t_lo && t1 < t_hi;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float o0[8], o1[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float d4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int p = 0; p < NK; ++p)
#pragma unroll
            for (int i = 0; i < P::A / NK; ++i) {
              const uint4 f = A[p * (P::A / NK) + i];
              mma_16816<F16>(d4, f.x, f.y, f.z, f.w, wb[p][4 * h + j][0], wb[p][4 * h + j][NE == 1 ? 0 : 1]);
            }
          o0[2 * j] = d4[0]; o0[2 * j + 1] = d4[1]; o1[2 * j] = d4[2]; o1[2 * j + 1] = d4[3];
        }
        uint32_t r0[4], r1[4];
        const uint32_t* q0 = reinterpret_cast<const uint32_t*>(&old[2 * h]);
        const uint32_t* q1 = reinterpret_cast<const uint32_t*>(&old[2 * h + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 f0 = make_float2(0.f, 0.f), f1 = f0;
          if (add) {
            f0 = H::unpack(q0[i]);
            f1 = H::unpack(q1[i]);
          }
          r0[i] = H::pack(fmaf(o0[2 * i], inv.x, f0.x), fmaf(o0[2 * i + 1], inv.x, f0.y));
          r1[i] = H::pack(fmaf(o1[2 * i], inv.y, f1.x), fmaf(o1[2 * i + 1], inv.y, f1.y));
        }
        if (v0) __stcs(reinterpret_cast<uint4*>(dx + (size_t)t0 * D + 32 * h), make_uint4(r0[0], r0[1], r0[2], r0[3]));
        if (v1) __stcs(reinterpret_cast<uint4*>(dx + (size_t)t1 * D + 32 * h), make_uint4(r1[0], r1[1], r1[2], r1[3]));
      }
    }
    if (b + S < b1) {                              // all that the stage held has been used: refill it
      copy_rows(b + S, st);
      copy_parts(b + S, st);
    }
    cp_commit();
    st = st + 1 == S ? 0 : st + 1;
  }
  cp_wait<0>();
  // the four ranges' sums, added in order.  Lane (g, c): expert row g (and g + 8), columns 16c + 8s + j
  __syncthreads();
  float* sum = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int p = 0; p < NK; ++p)
#pragma unroll
    for (int r = 0; r < (NE == 1 ? 1 : 2); ++r) {
      float* row = sum + ((size_t)w * EP + p * 16 + r * 8 + g) * 64 + 16 * c;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          row[8 * s + j] = NE == 1 ? acc[p][j][s] + acc[p][j][2 + s] : acc[p][j][2 * r + s];
    }
  __syncthreads();
  float* part = a.partials + (size_t)group * E * D + col;
  for (int i = threadIdx.x; i < E * 16; i += 128) {
    const int e = i >> 4, v = (i & 15) * 4;
    const float4* q = reinterpret_cast<const float4*>(sum + e * 64 + v);
    const float4 q0 = q[0], q1 = q[EP * 16], q2 = q[2 * EP * 16], q3 = q[3 * EP * 16];
    *reinterpret_cast<float4*>(part + (size_t)e * D + v) =
        make_float4((q0.x + q1.x) + (q2.x + q3.x), (q0.y + q1.y) + (q2.y + q3.y), (q0.z + q1.z) + (q2.z + q3.z),
                    (q0.w + q1.w) + (q2.w + q3.w));
  }
}

// ---------------------------------------------------------------- fp32
// FFMA throughout (a tensor core would round x).  One warp per TOK tokens: lane l holds columns
// 4l + 128 i of their rows and of Wg's.  TOK: four share each read of Wg where the tokens fill the
// device all the same, else one (T = 512: 18 us with four).
template <int EP, int TOK>
__global__ void __launch_bounds__(128) seq_scores_f32_kernel(SeqBalArgs a) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int D = a.D, E = a.E;
  const int tb = (blockIdx.x * 4 + w) * TOK;
  launch_dependents();
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  float l[TOK][EP];
#pragma unroll
  for (int i = 0; i < TOK; ++i)
#pragma unroll
    for (int e = 0; e < EP; ++e) l[i][e] = 0.f;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* x = static_cast<const float*>(a.x);
  const float* wg = static_cast<const float*>(a.wg);
#pragma unroll(EP * TOK <= 32 ? 3 : 1)
  for (int d = lane * 4; d < D; d += 128) {
    float4 xv[TOK];
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      const int t = tb + i;
      xv[i] = t < a.T ? __ldg(reinterpret_cast<const float4*>(x + (size_t)t * D + d)) : zero;
    }
#pragma unroll
    for (int e = 0; e < EP; ++e) {
      if (e < E) {
        const float4 wv = __ldg(reinterpret_cast<const float4*>(wg + (size_t)e * D + d));
#pragma unroll
        for (int i = 0; i < TOK; ++i)
          l[i][e] = fmaf(xv[i].x, wv.x, fmaf(xv[i].y, wv.y, fmaf(xv[i].z, wv.z, fmaf(xv[i].w, wv.w, l[i][e]))));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TOK; ++i)
#pragma unroll
    for (int e = 0; e < EP; ++e)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], o);
  // every lane holds every sum; lane e keeps expert e's
  grid_dependency_wait();
  const float aux = a.aux_scale / (float)max(*a.live, 1);
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
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
    if (t < a.T) {
      if (lane == 0) a.tok_loss[t] = tk.x >= 0 ? share : 0.f;
      if (a.grads && lane < EP) a.dl[(size_t)t * EP + lane] = tk.x >= 0 && lane < E ? P * (dp - pc) : 0.f;
    }
  }
}

// One block per (128 columns, four ranges of 16-token blocks), a warp to a range: lane l owns four
// columns, its slice of dWg in registers over the range.  D is a multiple of 64: half of a last slab
// may idle.  Four tokens' rows are loaded together.  Wg's columns stay in registers up to 8 experts.
template <int EP>
__global__ void __launch_bounds__(128) seq_grads_f32_kernel(SeqBalArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int U = EP == 32 ? 2 : 4;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int D = a.D, E = a.E;
  const int slabs = (D + 127) / 128, group = blockIdx.x / slabs, col = (blockIdx.x % slabs) * 128 + lane * 4;
  launch_dependents();
  const bool mine = col < D;
  const int range = group * 4 + w;
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  const int t_begin = max(range * a.blocks_per_range * 16, t_lo);
  const int t_end = min(min(a.T, t_hi), (range + 1) * a.blocks_per_range * 16);
  float4 acc[EP], wv[EP == 8 ? EP : 1];
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* x = static_cast<const float*>(a.x) + col;
  const float* wg = static_cast<const float*>(a.wg) + col;
  float* dx = a.dx ? static_cast<float*>(a.dx) + col : nullptr;
#pragma unroll
  for (int e = 0; e < EP; ++e) {
    acc[e] = zero;
    if (EP == 8) wv[e % (EP == 8 ? EP : 1)] = mine && e < E ? __ldg(reinterpret_cast<const float4*>(wg + (size_t)e * D)) : zero;
  }
  grid_dependency_wait();
  if (mine) {
    for (int tb = t_begin; tb < t_end; tb += U) {
      float4 xv[U], o[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = tb + u < t_end;
        xv[u] = in ? __ldg(reinterpret_cast<const float4*>(x + (size_t)(tb + u) * D)) : zero;
        o[u] = in && dx && a.accumulate ? *reinterpret_cast<const float4*>(dx + (size_t)(tb + u) * D) : zero;
      }
#pragma unroll
      for (int e4 = 0; e4 < EP; e4 += 4) {
        float4 dr[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          dr[u] = tb + u < t_end ? *reinterpret_cast<const float4*>(a.dl + (size_t)(tb + u) * EP + e4) : zero;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = e4 + i;
          if (e < E) {
            const float4 we = EP == 8 ? wv[e % (EP == 8 ? EP : 1)] : __ldg(reinterpret_cast<const float4*>(wg + (size_t)e * D));
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const float d = i == 0 ? dr[u].x : i == 1 ? dr[u].y : i == 2 ? dr[u].z : dr[u].w;
              acc[e].x = fmaf(d, xv[u].x, acc[e].x); acc[e].y = fmaf(d, xv[u].y, acc[e].y);
              acc[e].z = fmaf(d, xv[u].z, acc[e].z); acc[e].w = fmaf(d, xv[u].w, acc[e].w);
              o[u].x = fmaf(d, we.x, o[u].x); o[u].y = fmaf(d, we.y, o[u].y);
              o[u].z = fmaf(d, we.z, o[u].z); o[u].w = fmaf(d, we.w, o[u].w);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (dx && tb + u < t_end) *reinterpret_cast<float4*>(dx + (size_t)(tb + u) * D) = o[u];
    }
  }
  // the four ranges' sums, added in order
  float4* sum = reinterpret_cast<float4*>(ring);
#pragma unroll
  for (int e = 0; e < EP; ++e) sum[(w * EP + e) * 32 + lane] = acc[e];
  __syncthreads();
  float* part = a.partials + (size_t)group * E * D + (col - lane * 4);
  for (int i = threadIdx.x; i < E * 32; i += 128) {
    const int e = i >> 5, l = i & 31;
    if (col - lane * 4 + 4 * l >= D) continue;
    const float4 q0 = sum[e * 32 + l], q1 = sum[(EP + e) * 32 + l], q2 = sum[(2 * EP + e) * 32 + l], q3 = sum[(3 * EP + e) * 32 + l];
    *reinterpret_cast<float4*>(part + (size_t)e * D + 4 * l) =
        make_float4((q0.x + q1.x) + (q2.x + q3.x), (q0.y + q1.y) + (q2.y + q3.y), (q0.z + q1.z) + (q2.z + q3.z),
                    (q0.w + q1.w) + (q2.w + q3.w));
  }
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
// db sums `db_rows` rows of ep values: dl's own rows (fp32) or the scores kernel's sums of 16.
__global__ void __launch_bounds__(kFinThreads) seq_finish_kernel(SeqBalArgs a, const float* db_in, int db_rows, int ep,
                                                                 int wg_blocks, int db_blocks) {
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
    for (int k = w; k < a.groups; k += NW * 8)
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (k + u * NW < a.groups) r[u] += __ldcg(a.partials + (size_t)(k + u * NW) * stride + i);
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
    double s = 0.0;
#pragma unroll 4
    for (int k = tid; k < db_rows; k += kFinThreads) s += (double)__ldcg(db_in + (size_t)k * ep + blk);
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
  // whole blocks of 16 tokens by their sums, the rest token by token
  const int whole = a.blk_loss ? (lo + 15) / 16 : 0, end = a.blk_loss ? hi / 16 : 0;
  const int first = whole < end ? whole * 16 : hi, last = whole < end ? end * 16 : hi;
  double s = 0.0;
#pragma unroll 4
  for (int t = lo + tid; t < first; t += kFinThreads) s += (double)__ldcg(a.tok_loss + t);
#pragma unroll 4
  for (int b = whole + tid; b < end; b += kFinThreads) s += (double)__ldcg(a.blk_loss + b);
#pragma unroll 4
  for (int t = last + tid; t < hi; t += kFinThreads) s += (double)__ldcg(a.tok_loss + t);
  s = block_sum_f64(s, sh);
  if (tid == 0) {
    if (blk < a.n_seqs) a.seq_loss[blk] = (float)s;
    else *a.loss = (float)(s / (double)max(*a.live, 1));
  }
}

template <typename... P, typename... Q>
cudaError_t chained(void (*k)(P...), int grid, int threads, int smem, cudaStream_t s, Q... args) {
  if (smem > 32 * 1024) {                          // with what a kernel declares, above the default 48 KB
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
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
  cudaError_t e = chained(seq_scores_kernel<NE, F16>, (nblk + kScWarps - 1) / kScWarps, kScWarps * 32, kScSmem, s, a);
  if (e != cudaSuccess || !a.grads) return e;
  return chained(seq_grads_kernel<NE, F16>, a.D / 64 * a.groups, 128, GradRing<NE, F16>::Smem, s, a);
}
template <int EP>
cudaError_t launch32(const SeqBalArgs& a, cudaStream_t s) {
  cudaError_t e = a.T <= kSbF32Single ? chained(seq_scores_f32_kernel<EP, 1>, (a.T + 3) / 4, 128, 0, s, a)
                                      : chained(seq_scores_f32_kernel<EP, 4>, (a.T + 15) / 16, 128, 0, s, a);
  if (e != cudaSuccess || !a.grads) return e;
  return chained(seq_grads_f32_kernel<EP>, (a.D + 127) / 128 * a.groups, 128, EP * 2048, s, a);
}
template <bool F16>
cudaError_t launch16_e(const SeqBalArgs& a, cudaStream_t s) {
  return a.E <= 8 ? launch16<1, F16>(a, s) : a.E <= 16 ? launch16<2, F16>(a, s) : launch16<4, F16>(a, s);
}

}  // namespace

int seq_balance_ep(int E) { return E <= 8 ? 8 : E <= 16 ? 16 : 32; }

size_t seq_balance_frag_bytes(int E, int dtype) {
  const bool f16 = dtype == MOE_F16;
  const int n = E <= 8    ? (f16 ? Parts<1, true>::A + Parts<1, true>::T : Parts<1, false>::A + Parts<1, false>::T)
                : E <= 16 ? (f16 ? Parts<2, true>::A + Parts<2, true>::T : Parts<2, false>::A + Parts<2, false>::T)
                          : (f16 ? Parts<4, true>::A + Parts<4, true>::T : Parts<4, false>::A + Parts<4, false>::T);
  return (size_t)n * 512;
}

void seq_balance_plan(int T, int D, int E, int dtype, int* groups, int* blocks_per_range) {
  const int slabs = dtype == MOE_F32 ? (D + 127) / 128 : D / 64;
  const int nblk = (T + 15) / 16;
  int r = kSbSms * (E <= 16 ? 3 : 2) / slabs * 4;  // one wave of blocks, four ranges each
  if (r > nblk) r = nblk;
  if (r < 1) r = 1;
  *blocks_per_range = (nblk + r - 1) / r;
  const int ranges = *blocks_per_range > 0 ? (nblk + *blocks_per_range - 1) / *blocks_per_range : 0;
  *groups = (ranges + 3) / 4;
}

cudaError_t launch_seq_balance(const SeqBalArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const bool small = a.T <= kCountSmall && (long long)a.n_seqs * a.E <= kCountSmall && a.n_seqs < kOffSmem;
  if (small) {
    seq_count_kernel<true><<<1, 1024, 0, s>>>(a);
  } else {
    e = cudaMemsetAsync(a.counts, 0, (size_t)a.n_seqs * a.E * sizeof(int32_t), s);
    if (e == cudaSuccess && a.n_seqs >= kOffSmem) e = cudaMemsetAsync(a.live, 0, sizeof(int), s);
    if (e != cudaSuccess) return e;
    seq_count_kernel<false><<<(a.T + kCountThreads - 1) / kCountThreads, kCountThreads, 0, s>>>(a);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.dtype == MOE_F32)
    e = a.E <= 8 ? launch32<8>(a, s) : a.E <= 16 ? launch32<16>(a, s) : launch32<32>(a, s);
  else
    e = a.dtype == MOE_F16 ? launch16_e<true>(a, s) : launch16_e<false>(a, s);
  if (e != cudaSuccess) return e;
  const int wg_blocks = a.dwg ? a.E * a.D / 32 : 0, db_blocks = a.dbias ? a.E : 0;
  const bool f32 = a.dtype == MOE_F32;
  return chained(seq_finish_kernel, wg_blocks + db_blocks + a.n_seqs + 1, kFinThreads, 0, s, a,
                 (const float*)(f32 ? a.dl : a.db_part), f32 ? a.T : (a.T + 15) / 16, seq_balance_ep(a.E), wg_blocks, db_blocks);
}

}  // namespace moe
