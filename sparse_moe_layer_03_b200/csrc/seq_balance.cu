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
// x holds, and their dx stays; or, with all_gates, the part that their own dgate gives them (C = 0).
//
// The launches, chained by programmatic dependent launch:
//   count   sequence and factor of every token, counts (integer atomics; cleared before, where many)
//   scores  logits, softmax, dl: reads x once.  Its logits are formed while count runs
//   grads   dx and the partial sums of dWg: reads x again (from L2 where it fits), dx in and out
//   finish  the partial sums of dWg and db in a fixed order, the losses
// or, for 16-bit rows of 640 to 1152 and E <= 16, scores and grads as one kernel that reads x once (below;
// T = 32768, D = 1152, E = 8, dx added to: 48 us, 4.7 TB/s, against 23 + 43; the whole call 55 against 74).
//
// In the two kernels the mma.sync fragments are 16 consecutive bytes of a row in every lane.  Where an
// index is summed over (the columns in the logits) or names an output (the columns of dx and of
// dWg) the order in which a fragment holds it is free, so each lane copies the pieces of rows that
// will be its own fragments and reads back only what it copied: a ring of cp.async stages that needs
// no barrier, no swizzle and no ldmatrix, and keeps kilobytes of each warp in flight.  dWg sums over
// tokens, whose pairs lie in different rows: two rows' pieces are interleaved in registers.
// dl goes between the kernels already in fragment order, as it is and transposed (movmatrix), in
// 16-bit parts that add up to it: for dx two; for dWg, which stays in fp32, three of bf16 (24 bits)
// or two of fp16 (22 bits below the largest of its expert's 16: a scale for each expert, so that the
// gate row of one hardly ever chosen keeps its digits; for dx a scale for each token).
// With E <= 8 two parts share one k16 step.
#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kCountThreads = 256;
constexpr int kOffSmem = 2048;                     // offsets kept in shared memory up to this many
constexpr int kOneThreads = 1024;
constexpr int kOneTokens = 2048, kOneCounts = 4096;   // most tokens and counts of the one-block form
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
// first and one past the last row that take part: those of the sequences, or all
__device__ __forceinline__ void live_rows(const SeqBalArgs& a, int& lo, int& hi) {
  const bool some = a.offsets && !a.all_gates;
  lo = some ? min(max(a.offsets[0], 0), a.T) : 0;
  hi = some ? min(max(a.offsets[a.n_seqs], lo), a.T) : a.T;
}
__device__ __forceinline__ int slots_of(const SeqBalArgs& a, int t) {
  return a.n_sel ? min(max(a.n_sel[t], 0), a.Kmax) : a.K;
}

// ---------------------------------------------------------------- count
// Counts (and the number of sequences that hold a row) to zero, ahead of the count kernel, which is set up
// and has found its tokens' sequences by the time it ends (a memset would be waited for).
__global__ void __launch_bounds__(kCountThreads) seq_clear_kernel(int32_t* counts, long long n, int* live) {
  launch_dependents();
  for (long long i = (long long)blockIdx.x * kCountThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kCountThreads)
    counts[i] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *live = 0;
}

// One thread per token: its sequence by binary search, its selected experts into the counts.  ONE: one
// block, the counts in shared memory; no clearing, no global atomics.  Else equal (sequence, expert) keys of
// a warp are merged (as in the frequency kernel) and added to counts that were cleared before.  The choice
// is by the tokens: a cluster of eight blocks adding up their shared memory took 9.3 us for 32768 tokens
// (half of it more blocks' work: 128 blocks and clearing 6.5), and gained nothing from 10000 down.
template <bool ONE>
__global__ void __launch_bounds__(ONE ? kOneThreads : kCountThreads) seq_count_kernel(SeqBalArgs a) {
  __shared__ int off_s[kOffSmem];
  __shared__ int hist[ONE ? kOneCounts : 1];
  __shared__ int full_s;
  launch_dependents();
  const int tid = threadIdx.x, n = a.n_seqs, nt = blockDim.x;
  constexpr int kAhead = 4;                        // slots loaded with the token
  const int* off = a.offsets;
  const bool in_smem = n + 1 <= kOffSmem;
  if (ONE)
    for (int i = tid; i < n * a.E; i += nt) hist[i] = 0;
  if (tid == 0) full_s = 0;
  if (off && in_smem) {
    for (int i = tid; i <= n; i += nt) off_s[i] = off[i];
    off = off_s;
  }
  // a round: kRound tokens of the thread, their slots on the way together (the first round's beside the offsets)
  constexpr int kRound = ONE ? 2 : 1;
  const int stride = gridDim.x * nt;
  int ns[kRound], idx[kRound][kAhead];
  auto load_slots = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kRound; ++i) {
      const int t = t0 + i * stride;
      ns[i] = t < a.T ? slots_of(a, t) : 0;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) idx[i][k] = t < a.T && k < a.Kmax ? a.topk_idx[(size_t)t * a.Kmax + k] : -1;
    }
  };
  load_slots(blockIdx.x * nt + tid);
  __syncthreads();
  if (!ONE) grid_dependency_wait();                // the counts are clear
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
  for (int first = blockIdx.x * nt; first < a.T; first += kRound * stride) {
#pragma unroll
    for (int i = 0; i < kRound; ++i) {
      const int t = first + i * stride + tid;
      int sid = -1, len = 0;
      if (t < a.T) {
        if (off) {
          int lo = 0, hi = n;                      // the last sequence that starts at or before t
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
        const float coef = sid >= 0 ? a.factor / ((float)len * (float)len) : 0.f;
        a.tok[t] = make_int2(sid, __float_as_int(coef));
      }
      const int use = sid >= 0 || a.all_gates ? ns[i] : 0;
      auto add = [&](int k, int e) {               // every lane, for __match_any_sync
        long long key = -1;
        if (k < use) {
          if (e >= a.E) set_status(a.status, DEV_BAD_INDEX, 411);
          else if (e >= 0 && sid >= 0) key = (long long)sid * a.E + e;
        }
        if (ONE) {
          if (key >= 0) atomicAdd(&hist[key], 1);
        } else {
          const unsigned same = __match_any_sync(0xffffffffu, key);
          if (key >= 0 && (tid & 31) == __ffs(same) - 1) atomicAdd(&a.counts[key], __popc(same));
        }
      };
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k < a.Kmax) add(k, idx[i][k]);
      for (int k = kAhead; k < a.Kmax; ++k) {
        if (!__any_sync(0xffffffffu, k < use)) break;
        add(k, k < use ? a.topk_idx[(size_t)t * a.Kmax + k] : -1);
      }
    }
    if (first + kRound * stride < a.T) load_slots(first + kRound * stride + tid);
  }
  __syncthreads();
  if (ONE)
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
  static constexpr int V = !F16 ? 0 : NE == 4 ? 2 : 1;      // float4s of inverse scales for each row pair
};
// fp16's inverse scales of a 16-token block, as lane (g, c) takes them: of rows g and g + 8, and of experts
// 8 nt + g.
template <int NE> struct DlScales {
  float row[2] = {1.f, 1.f}, expert[NE];
  __device__ __forceinline__ void store(float4* p) const {
    p[0] = make_float4(row[0], row[1], NE < 4 ? expert[0] : 0.f, NE == 2 ? expert[1 % NE] : 0.f);
    if (NE == 4) p[1] = make_float4(expert[0], expert[1 % NE], expert[2 % NE], expert[3 % NE]);
  }
  __device__ __forceinline__ void load(const float4& u, const float4& v) {
    row[0] = u.x;
    row[1] = u.y;
    const float e[4] = {NE == 4 ? v.x : u.z, NE == 4 ? v.y : u.w, v.z, v.w};
#pragma unroll
    for (int nt = 0; nt < NE; ++nt) expert[nt] = e[nt];
  }
};

// The gates' gradients of a 16-token block, lane l < 16 holding token l's first slots: loaded ahead of
// their use.
struct GatesAhead {
  int ns, e[kGateAhead];
  float v[kGateAhead];
};
__device__ __forceinline__ GatesAhead load_gates(const SeqBalArgs& a, int rb) {
  GatesAhead q;
  const int lane = threadIdx.x & 31, t = rb * 16 + lane;
  const bool in = a.dgate && lane < 16 && t < a.T;
  q.ns = in ? slots_of(a, t) : 0;
#pragma unroll
  for (int k = 0; k < kGateAhead; ++k) {
    q.e[k] = in && k < a.Kmax ? a.topk_idx[(size_t)t * a.Kmax + k] : -1;
    q.v[k] = in && k < a.Kmax ? a.dgate[(size_t)t * a.Kmax + k] : 0.f;
  }
  return q;
}
// ... scattered to their experts, each token by one lane: dp [16][ep] in shared memory
template <int EP>
__device__ __forceinline__ void scatter_gates(const SeqBalArgs& a, const GatesAhead& q, int rb, int t_lo, int t_hi, float* dp) {
  const int lane = threadIdx.x & 31, t = rb * 16 + lane;
  __syncwarp();
  for (int i = lane; i < 16 * EP; i += 32) dp[i] = 0.f;
  __syncwarp();
  if (t >= t_lo && t < t_hi) {                     // ns = 0 on the other lanes
#pragma unroll
    for (int k = 0; k < kGateAhead; ++k)
      if (k < q.ns && q.e[k] >= 0 && q.e[k] < a.E) dp[lane * EP + q.e[k]] += q.v[k];
    for (int k = kGateAhead; k < q.ns; ++k) {
      const int e = a.topk_idx[(size_t)t * a.Kmax + k];
      if (e >= 0 && e < a.E) dp[lane * EP + e] += a.dgate[(size_t)t * a.Kmax + k];
    }
  }
  __syncwarp();
}

// What a lane holds of a block: rows t0 = 16 rb + g and t0 + 8 (r = 0, 1), experts nt * 8 + 2c + q.
template <int NE> using RowPair = float[2][NE][2];

// C = factor * counts of the rows' sequences; in: the row takes part
template <int NE>
__device__ __forceinline__ void load_counts(const SeqBalArgs& a, const bool* live, int t0, RowPair<NE>& C, bool* in) {
  const int c = threadIdx.x & 3;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int2 tk = live[r] ? a.tok[t0 + 8 * r] : make_int2(-1, 0);
    in[r] = tk.x >= 0 || (live[r] && a.all_gates);
#pragma unroll
    for (int nt = 0; nt < NE; ++nt)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int e = nt * 8 + 2 * c + q;
        C[r][nt][q] = tk.x >= 0 && e < a.E ? __int_as_float(tk.y) * (float)a.counts[(size_t)tk.x * a.E + e] : 0.f;
      }
  }
}

// Logits (without the bias) to dl in place; the tokens' and the block's shares of the loss are written.
template <int NE>
__device__ __forceinline__ void logits_to_dl(const SeqBalArgs& a, int rb, const float* dp_s, float aux, const RowPair<NE>& C,
                                             const bool* in, RowPair<NE>& l) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, E = a.E;
  float loss16 = 0.f;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float m = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NE; ++nt)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int e = nt * 8 + 2 * c + q;
        l[r][nt][q] = e < E ? l[r][nt][q] + (a.bias ? __ldg(a.bias + e) : 0.f) : -INFINITY;
        m = fmaxf(m, l[r][nt][q]);
      }
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
    float dp[NE][2], share = 0.f, pc = 0.f;
#pragma unroll
    for (int nt = 0; nt < NE; ++nt)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        l[r][nt][q] *= iz;
        share += l[r][nt][q] * C[r][nt][q];
        dp[nt][q] = aux * C[r][nt][q] + (a.dgate ? dp_s[(g + 8 * r) * NE * 8 + nt * 8 + 2 * c + q] : 0.f);
        pc += l[r][nt][q] * dp[nt][q];
      }
    share = quad_sum(share);
    pc = quad_sum(pc);
    share = in[r] ? share : 0.f;
    const int t = rb * 16 + g + 8 * r;
    if (c == 0 && t < a.T) a.tok_loss[t] = share;
    loss16 += share;
#pragma unroll
    for (int nt = 0; nt < NE; ++nt)
#pragma unroll
      for (int q = 0; q < 2; ++q) l[r][nt][q] = in[r] ? l[r][nt][q] * (dp[nt][q] - pc) : 0.f;
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) loss16 += __shfl_xor_sync(0xffffffffu, loss16, o);
  if (lane == 0 && rb * 16 < a.T) a.blk_loss[rb] = loss16;
}

// dl in fragment order: fa (k = experts) for dx, ft (k = tokens, by movmatrix) for dWg, and fp16's inverse
// scales.
template <int NE, bool F16>
__device__ __forceinline__ void dl_fragments(const RowPair<NE>& dl, uint4* fa, uint4* fw, DlScales<NE>& scale) {
  using H = H16<F16>;
  using P = Parts<NE, F16>;
  float sr[2] = {1.f, 1.f}, se[NE][2];
  if (F16) {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mr = 0.f;
#pragma unroll
      for (int nt = 0; nt < NE; ++nt) mr = fmaxf(mr, fmaxf(fabsf(dl[r][nt][0]), fabsf(dl[r][nt][1])));
      sr[r] = pow2_scale(quad_max(mr), scale.row[r]);
    }
#pragma unroll
    for (int nt = 0; nt < NE; ++nt) {
      float inv[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float me = fmaxf(fabsf(dl[0][nt][q]), fabsf(dl[1][nt][q]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) me = fmaxf(me, __shfl_xor_sync(0xffffffffu, me, o));
        se[nt][q] = pow2_scale(me, inv[q]);
      }
      // expert 8 nt + g is a lane's with c = g / 2
      const float even = __shfl_sync(0xffffffffu, inv[0], g >> 1), odd = __shfl_sync(0xffffffffu, inv[1], g >> 1);
      scale.expert[nt] = g & 1 ? odd : even;
    }
  }
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
      if (F16) split(dl[r][nt][0] * se[nt][0], dl[r][nt][1] * se[nt][1], &ft[r][0][nt], NE);
#pragma unroll
      for (int i = 0; i < NP; ++i) ft[r][i][nt] = movm_t(F16 ? ft[r][i][nt] : f[r][i][nt]);
    }
  if (NE == 1) {                                   // k (or m) = 0..7 the first part, 8..15 the second; then the third
    fa[0] = make_uint4(f[0][0][0], f[1][0][0], f[0][1][0], f[1][1][0]);
    fw[0] = make_uint4(ft[0][0][0], ft[0][1][0], ft[1][0][0], ft[1][1][0]);
    if (NP == 3) fw[P::T - 1] = make_uint4(ft[0][NP - 1][0], 0u, ft[1][NP - 1][0], 0u);
  } else {
#pragma unroll
    for (int p = 0; p < P::NK; ++p)
#pragma unroll
      for (int i = 0; i < NP; ++i) {               // 16 experts: part after part
        constexpr int o = NE > 1;
        if (i < 2) fa[2 * p + i] = make_uint4(f[0][i][2 * p], f[1][i][2 * p], f[0][i][2 * p + o], f[1][i][2 * p + o]);
        fw[NP * p + i] = make_uint4(ft[0][i][2 * p], ft[0][i][2 * p + o], ft[1][i][2 * p], ft[1][i][2 * p + o]);
      }
  }
}

// One warp per 16 tokens.  NE: 8-expert tiles of the logits.  In a k32 step lane (g, c) (g = lane / 4,
// c = lane % 4) holds columns 8c .. 8c+7 of rows g and g + 8 of x and of row g of each 8 rows of Wg:
// the first four of them serve as k = 2c, 2c+1, 2c+8, 2c+9 of one k16 product, the others of a second.
template <int NE, bool F16>
__global__ void __launch_bounds__(kScWarps * 32) seq_scores_kernel(SeqBalArgs a) {
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
  const GatesAhead gates = load_gates(a, rb);      // on their way meanwhile
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  const bool live[2] = {t0 >= t_lo && t0 < t_hi, t1 >= t_lo && t1 < t_hi};
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
  RowPair<NE> l, C;
#pragma unroll
  for (int nt = 0; nt < NE; ++nt)
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int r = 0; r < 2; ++r) l[r][nt][q] = acc[nt][0][2 * r + q] + acc[nt][1][2 * r + q];
  if (a.dgate) scatter_gates<EP>(a, gates, rb, t_lo, t_hi, &dp_s[w][0][0]);
  grid_dependency_wait();                          // from here on: what count wrote
  bool in[2];
  load_counts<NE>(a, live, t0, C, in);
  logits_to_dl<NE>(a, rb, &dp_s[w][0][0], a.aux_scale / (float)max(*a.live, 1), C, in, l);
  if (!a.grads || rb * 16 >= a.T) return;
  // db of the 16 tokens
#pragma unroll
  for (int nt = 0; nt < NE; ++nt)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float sum = l[0][nt][q] + l[1][nt][q];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (g == 0) a.db_part[(size_t)rb * EP + nt * 8 + 2 * c + q] = sum;
    }
  using P = Parts<NE, F16>;
  uint4 fa[P::A], fw[P::T];
  DlScales<NE> scale;
  dl_fragments<NE, F16>(l, fa, fw, scale);
  if (F16 && c == 0) scale.store(a.scales + ((size_t)rb * 8 + g) * P::V);
  uint4* out = a.frag + (size_t)rb * (P::A + P::T) * 32 + lane;
#pragma unroll
  for (int i = 0; i < P::A; ++i) out[i * 32] = fa[i];
#pragma unroll
  for (int i = 0; i < P::T; ++i) out[(P::A + i) * 32] = fw[i];
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
  static constexpr int Slots = 8 + P::A + P::T + P::V;            // 512 bytes each: x 4, dx 4, dl, scales
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
#pragma unroll
    for (int i = 0; i < P::V; ++i) cp16(dst + (P::A + P::T + i) * 512, a.scales + ((size_t)b * 8 + g) * P::V + i, true);
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
    DlScales<NE> inv;
    if (F16) {
      const float4* s = reinterpret_cast<const float4*>(in + (8 + P::A + P::T) * 512);
      inv.load(s[0], s[32 * (P::V > 1)]);          // the second, where there is one, 512 bytes on
    }
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
        for (int q = 0; q < 4; ++q)
          acc[p][j][q] = F16 ? fmaf(d4[q], inv.expert[NE == 1 ? 0 : 2 * p + (q >> 1)], acc[p][j][q]) : acc[p][j][q] + d4[q];
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
          r0[i] = H::pack(fmaf(o0[2 * i], inv.row[0], f0.x), fmaf(o0[2 * i + 1], inv.row[0], f0.y));
          r1[i] = H::pack(fmaf(o1[2 * i], inv.row[1], f1.x), fmaf(o1[2 * i + 1], inv.row[1], f1.y));
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

// ---------------------------------------------------------------- scores and grads in one, 16-bit types
// One block of 15 warps an SM over every grid-th 16-token block; x comes in once, by TMA, into a ring of
// whole blocks of rows (64-column boxes, 128-byte swizzle) and leaves it when both halves are done:
//   3 router warps, a token block each in turn: logits (ldmatrix and mma.sync on the stage), softmax, dl,
//     left in shared memory in fragment order;
//   12 column warps, each a slice of 32-column groups over all the block's tokens: dWg in registers from
//     the stage (transposed ldmatrix), dx from dl and the gate weight's columns in registers.
// They meet on mbarriers only (dl full and empty by router, x full by stage); the last column warp to leave
// a stage refills it.  For E <= 16 and rows of 640 (narrower ones leave the column warps too little: the two
// kernels' many independent warps hide latency better) to 1152.
constexpr int kFuRouters = 3, kFuCols = 12, kFuThreads = (kFuRouters + kFuCols) * 32;
constexpr int kFuGroups = 3;                       // 32-column groups a column warp holds
// The narrowest row.  One kernel against two, bf16, E = 8, whole calls replayed from a graph (us): at T = 32768
// 37.6 / 33.4 at D = 512, 39.4 / 35.8 at 576, 38.6 / 38.1 at 640, 40.0 / 41.1 at 704, 52.5 / 67.1 at 1152; at T = 8192
// 18.3 / 18.3, 19.0 / 19.1, 18.6 / 19.8, 19.3 / 21.5, 22.4 / 27.5; at T = 512 10.9 / 11.2, 11.1 / 11.6, 11.3 / 12.0,
// 11.4 / 12.4, 13.4 / 15.7.  Below 640 the two win by up to 4 us where calls are large, the one by up to 0.5
// where they are small.  16 experts cross a little later (T = 32768: 46.1 / 43.7 at 640, 49.4 / 50.7 at 768), with
// inputs out of L2 earlier (45.6 / 50.2 at 640, E = 8; 52.2 / 54.3, E = 16).
constexpr int kFuMinD = 640;
constexpr int kFuMaxStages = 6;
constexpr int kFuMaxSmem = 232448;

struct FusedSmem { int wg_stride, x, wg, dl, dl_slot, dp, old, misc, total, stage; };
// most 32-column groups a column warp holds
__host__ __device__ inline int fused_groups(int D) { return (D / 32 + kFuCols - 1) / kFuCols; }
// `held`: blocks whose slices of dx, to be added to, are on their way (0: dx is not added to)
__host__ __device__ inline FusedSmem fused_smem(int D, int ne, int frags, int stages, int held) {
  FusedSmem L;
  L.stage = 16 * D * 2;
  L.wg_stride = D * 2 + 16;
  L.dl_slot = frags * 512 + 128;
  L.x = 0;
  L.wg = stages * L.stage;
  L.dl = L.wg + ne * 8 * L.wg_stride;
  L.dp = L.dl + kFuRouters * L.dl_slot;
  L.old = L.dp + kFuRouters * 16 * ne * 8 * 4;
  L.misc = L.old + held * kFuCols * fused_groups(D) * 1024;
  L.total = L.misc + 256 + 1024;                   // barriers and counters; alignment of the stages
  return L;
}
// Stages of x and blocks of dx in flight.  Two blocks of dx where three stages fit beside them, else one:
// XL with 8 experts 57.5 us with (3, 2) against 62.5 with (4, 1); with 16, 88.3 with (2, 2) against 72.7
// with (3, 1).
struct FusedPlan { int stages, held; };
__host__ inline FusedPlan fused_plan(int D, int ne, int frags, bool add) {
  for (int held = add ? 2 : 0;; --held) {
    int n = kFuMaxStages;
    while (n > 0 && fused_smem(D, ne, frags, n, held).total > kFuMaxSmem) --n;
    if (n >= 3 || held <= 1) return {n, held};
  }
}

// Bounded wait until `need` loads have been issued into a stage.  A router may be a whole turn of the ring
// ahead, and a parity cannot tell its phase from the one two before: once the load is issued the phases
// before it are over, and the parity is unambiguous.
__device__ __forceinline__ bool wait_issued(volatile int* loads, int need, volatile int* abort_flag, int* status, int where) {
  if (*loads >= need) return true;
  const uint64_t t0 = global_ns();
#pragma unroll 1
  while (*loads < need) {
    if (*abort_flag) return false;
    __nanosleep(64);                               // the column warps need the issue slots
    if (global_ns() - t0 > kWaitLimitNs) {
      set_status(status, DEV_TIMEOUT, where);
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

template <int NE, bool F16>
__global__ void __launch_bounds__(kFuThreads, 1)
seq_fused_kernel(const __grid_constant__ CUtensorMap tmap_x, const SeqBalArgs a, const int stages, const int held_blocks) {
  using H = H16<F16>;
  using P = Parts<NE, F16>;
  constexpr int EP = NE * 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const bool add = held_blocks > 0;
  const FusedSmem L = fused_smem(a.D, NE, P::A + P::T, stages, held_blocks);
  const int D = a.D, E = a.E, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int g = lane >> 2, c = lane & 3, li = lane >> 3, lj = lane & 7;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.misc);
  uint64_t* dl_full = full + kFuMaxStages;
  uint64_t* dl_empty = dl_full + kFuRouters;
  uint64_t* wbar = dl_empty + kFuRouters;
  int* done = reinterpret_cast<int*>(wbar + 1);    // column warps that left a stage
  volatile int* loads = done + kFuMaxStages;       // loads issued into a stage
  volatile int* abort_flag = loads + kFuMaxStages;
  launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kFuMaxStages; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      done[i] = 0;
      loads[i] = 0;
    }
    for (int i = 0; i < kFuRouters; ++i) {
      mbar_init(smem_u32(&dl_full[i]), 1);
      mbar_init(smem_u32(&dl_empty[i]), kFuCols);
    }
    mbar_init(smem_u32(wbar), 1);
    *abort_flag = 0;
    fence_barrier_init();
    mbar_arrive_expect_tx(smem_u32(wbar), (uint32_t)(E * D * 2));
    for (int e = 0; e < E; ++e)
      bulk_load(smem_u32(smem + L.wg + e * L.wg_stride), static_cast<const uint8_t*>(a.wg) + (size_t)e * D * 2, (uint32_t)(D * 2),
                smem_u32(wbar));
  }
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  const int b_lo = t_lo / 16, b_hi = t_hi > t_lo ? (t_hi + 15) / 16 : b_lo;
  const int nb = b_hi - b_lo > (int)blockIdx.x ? (b_hi - b_lo - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0;
  auto block_of = [&](int j) { return b_lo + (int)blockIdx.x + j * (int)gridDim.x; };
  auto issue = [&](int j) {                        // one thread: block j into its stage
    const int st = j % stages;
    const uint32_t bar = smem_u32(&full[st]);
    loads[st] = loads[st] + 1;
    mbar_arrive_expect_tx(bar, (uint32_t)L.stage);
    tma_load_3d(smem_u32(smem + L.x + st * L.stage), &tmap_x, 0, block_of(j) * 16, 0, bar);
  };
  if (tid == 0)
    for (int j = 0; j < stages && j < nb; ++j) issue(j);
  for (int i = tid; i < (EP - E) * (D / 8); i += kFuThreads)   // rows of no expert
    *reinterpret_cast<uint4*>(smem + L.wg + (E + i / (D / 8)) * L.wg_stride + (i % (D / 8)) * 16) = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  int* status = a.status;
  if (w < kFuRouters) {
    // ------------------------------------------------ router warps
    const uint32_t wg = smem_u32(smem + L.wg);
    uint8_t* slot = smem + L.dl + w * L.dl_slot;
    float* dp = reinterpret_cast<float*>(smem + L.dp) + w * 16 * EP;
    float db[NE][2];
#pragma unroll
    for (int nt = 0; nt < NE; ++nt) db[nt][0] = db[nt][1] = 0.f;
    bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(wbar), 0, abort_flag, status, 420));
    bool waited = false;
    float aux = 0.f;
    for (int j = w; j < nb && ok; j += kFuRouters) {
      const int rb = block_of(j), st = j % stages, t0 = rb * 16 + g;
      const GatesAhead gates = load_gates(a, rb);
      const bool live[2] = {t0 >= t_lo && t0 < t_hi, t0 + 8 >= t_lo && t0 + 8 < t_hi};
      RowPair<NE> l, C;
      bool in[2];
      if (waited) load_counts<NE>(a, live, t0, C, in);
      ok = wait_issued(&loads[st], j / stages + 1, abort_flag, status, 427) &&
           mbar_wait(smem_u32(&full[st]), (j / stages) & 1, abort_flag, status, 421);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t xs = smem_u32(smem + L.x + st * L.stage);
      float acc[NE][4 / NE][4];                    // independent sums, to be added
#pragma unroll
      for (int nt = 0; nt < NE; ++nt)
#pragma unroll
        for (int u = 0; u < 4 / NE; ++u)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[nt][u][q] = 0.f;
#pragma unroll 2
      for (int box = 0; box < D / 64; ++box) {     // four k16 steps
        uint32_t b[NE][4][2];
        if (NE == 1) {
          ldsm_x4(wg + lj * L.wg_stride + box * 128 + li * 16, b[0][0][0], b[0][0][1], b[0][1][0], b[0][1][1]);
          ldsm_x4(wg + lj * L.wg_stride + box * 128 + 64 + li * 16, b[0][2][0], b[0][2][1], b[0][3][0], b[0][3][1]);
        } else {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            ldsm_x4(wg + ((li >> 1) * 8 + lj) * L.wg_stride + box * 128 + ks * 32 + (li & 1) * 16, b[0][ks][0], b[0][ks][1],
                    b[NE - 1][ks][0], b[NE - 1][ks][1]);
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const int row = (li & 1) * 8 + lj, chunk = ks * 2 + (li >> 1);
          uint32_t a0, a1, a2, a3;
          ldsm_x4(xs + box * 2048 + row * 128 + ((chunk ^ (row & 7)) << 4), a0, a1, a2, a3);
#pragma unroll
          for (int nt = 0; nt < NE; ++nt) mma_16816<F16>(acc[nt][ks % (4 / NE)], a0, a1, a2, a3, b[nt][ks][0], b[nt][ks][1]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NE; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float v = acc[nt][0][2 * r + q];
#pragma unroll
            for (int u = 1; u < 4 / NE; ++u) v += acc[nt][u][2 * r + q];
            l[r][nt][q] = v;
          }
      if (a.dgate) scatter_gates<EP>(a, gates, rb, t_lo, t_hi, dp);
      if (!waited) {                               // from here on: what count wrote
        grid_dependency_wait();
        waited = true;
        aux = a.aux_scale / (float)max(*a.live, 1);
        load_counts<NE>(a, live, t0, C, in);
      }
      logits_to_dl<NE>(a, rb, dp, aux, C, in, l);
#pragma unroll
      for (int nt = 0; nt < NE; ++nt)
#pragma unroll
        for (int q = 0; q < 2; ++q) db[nt][q] += l[0][nt][q] + l[1][nt][q];
      uint4 fa[P::A], fw[P::T];
      DlScales<NE> scale;
      dl_fragments<NE, F16>(l, fa, fw, scale);
      const int use = j / kFuRouters;
      if (use > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&dl_empty[w]), (use - 1) & 1, abort_flag, status, 422));
        if (!ok) break;
      }
      uint4* out = reinterpret_cast<uint4*>(slot) + lane;
#pragma unroll
      for (int i = 0; i < P::A; ++i) out[i * 32] = fa[i];
#pragma unroll
      for (int i = 0; i < P::T; ++i) out[(P::A + i) * 32] = fw[i];
      if (F16 && c == 0) scale.store(reinterpret_cast<float4*>(slot + (P::A + P::T) * 512) + g);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&dl_full[w]));
    }
    if (!waited) grid_dependency_wait();
#pragma unroll
    for (int nt = 0; nt < NE; ++nt)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float sum = db[nt][q];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (g == 0) a.db_part[((size_t)blockIdx.x * kFuRouters + w) * EP + nt * 8 + 2 * c + q] = sum;
      }
  } else {
    // ------------------------------------------------ column warps
    const int cw = w - kFuRouters, groups = D / 32;
    const int g0 = cw * groups / kFuCols, g1 = (cw + 1) * groups / kFuCols;
    uint32_t wb[kFuGroups][4][NE];                 // gate weight fragments of dx: rows e = 8h + 2c, + 1
    const uint16_t* wg = static_cast<const uint16_t*>(a.wg);
    float acc[kFuGroups][4][4];
#pragma unroll
    for (int gi = 0; gi < kFuGroups; ++gi)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[gi][j][q] = 0.f;
#pragma unroll
        for (int h = 0; h < NE; ++h) {
          const int e = h * 8 + 2 * c, d = (g0 + gi) * 32 + 8 * (g >> 1) + 2 * j + (g & 1);
          const uint32_t u = g0 + gi < g1 && e < E ? wg[(size_t)e * D + d] : 0u;
          const uint32_t v = g0 + gi < g1 && e + 1 < E ? wg[(size_t)(e + 1) * D + d] : 0u;
          wb[gi][j][h] = u | (v << 16);
        }
      }
    uint16_t* dx = static_cast<uint16_t*>(a.dx) + g0 * 32 + 8 * c;
    const int gmax = fused_groups(D);
    const uint8_t* held = smem + L.old + cw * held_blocks * gmax * 1024 + lane * 16;
    auto copy_old = [&](int j) {                   // what dx holds of block j, this lane's own pieces
      if (add && j < nb) {
        const int t0 = block_of(j) * 16 + g, t1 = t0 + 8;
        const bool v0 = t0 >= t_lo && t0 < t_hi, v1 = t1 >= t_lo && t1 < t_hi;
        const uint32_t dst = smem_u32(held) + (j & (held_blocks - 1)) * gmax * 1024;
        for (int gi = 0; gi < g1 - g0; ++gi) {
          cp16(dst + gi * 1024, dx + (v0 ? (size_t)t0 * D : 0) + gi * 32, v0);
          cp16(dst + gi * 1024 + 512, dx + (v1 ? (size_t)t1 * D : 0) + gi * 32, v1);
        }
      }
      cp_commit();
    };
    copy_old(0);
    if (held_blocks == 2) copy_old(1);
    bool ok = true;
    for (int j = 0; j < nb; ++j) {
      const int rb = block_of(j), st = j % stages, t0 = rb * 16 + g, t1 = t0 + 8;
      const bool v0 = t0 >= t_lo && t0 < t_hi, v1 = t1 >= t_lo && t1 < t_hi;
      const int r = j % kFuRouters;
      ok = mbar_wait(smem_u32(&dl_full[r]), (j / kFuRouters) & 1, abort_flag, status, 423) &&
           mbar_wait(smem_u32(&full[st]), (j / stages) & 1, abort_flag, status, 424);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint8_t* old = held + (add ? (j & (held_blocks - 1)) * gmax * 1024 : 0);
      const uint32_t xs = smem_u32(smem + L.x + st * L.stage);
      const uint8_t* slot = smem + L.dl + r * L.dl_slot;
      uint4 At[P::T];
#pragma unroll
      for (int i = 0; i < P::T; ++i) At[i] = reinterpret_cast<const uint4*>(slot)[(P::A + i) * 32 + lane];
      DlScales<NE> inv;
      if (F16) {
        const float4 s = reinterpret_cast<const float4*>(slot + (P::A + P::T) * 512)[g];
        inv.load(s, s);
      }
      // rows of no sequence may hold anything: their x counts as zero (tokens 2c, 2c+1 and 2c+8, 2c+9)
      const bool whole = rb * 16 >= t_lo && rb * 16 + 16 <= t_hi;
      uint32_t k0 = 0xffffffffu, k1 = 0xffffffffu;
      if (!whole) {
        auto live = [&](int i) { return rb * 16 + i >= t_lo && rb * 16 + i < t_hi; };
        k0 = (live(2 * c) ? 0xffffu : 0u) | (live(2 * c + 1) ? 0xffff0000u : 0u);
        k1 = (live(2 * c + 8) ? 0xffffu : 0u) | (live(2 * c + 9) ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int gi = 0; gi < kFuGroups; ++gi) {
        if (g0 + gi < g1) {
          // ---- dWg += dl^T x: two tiles of 8 columns at a time
          const int col = (g0 + gi) * 32;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = (li & 1) * 8 + lj, chunk = ((col & 63) >> 3) + 2 * h + (li >> 1);
            uint32_t b[2][2];
            ldsm_x4_t(xs + (col >> 6) * 2048 + t * 128 + ((chunk ^ (t & 7)) << 4), b[0][0], b[0][1], b[1][0], b[1][1]);
            if (!whole) {
              b[0][0] &= k0; b[1][0] &= k0;
              b[0][1] &= k1; b[1][1] &= k1;
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {          // the block's product, smallest part first, then one addition
              float d4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = P::T - 1; i >= 0; --i) mma_16816<F16>(d4, At[i].x, At[i].y, At[i].z, At[i].w, b[q][0], b[q][1]);
              float* s4 = acc[gi][2 * h + q];
#pragma unroll
              for (int k = 0; k < 4; ++k) s4[k] = F16 ? fmaf(d4[k], inv.expert[NE == 1 ? 0 : k >> 1], s4[k]) : s4[k] + d4[k];
            }
          }
        }
      }
      // this warp is done with x: the last one to leave the stage refills it
      __syncwarp();
      if (lane == 0) {
        __threadfence_block();
        if (atomicAdd(&done[st], 1) == kFuCols - 1) {
          done[st] = 0;
          if (j + stages < nb) {
            fence_async_shared();
            issue(j + stages);
          }
        }
      }
      // ---- dx (+)= dl Wg
      if (a.dx) {
        uint4 A[P::A];
#pragma unroll
        for (int i = 0; i < P::A; ++i) A[i] = reinterpret_cast<const uint4*>(slot)[i * 32 + lane];
        if (held_blocks == 2) cp_wait<1>();
        else if (held_blocks == 1) cp_wait<0>();
#pragma unroll
        for (int gi = 0; gi < kFuGroups; ++gi) {
          if (g0 + gi < g1) {
            float o0[8], o1[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float d4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = 0; i < P::A; ++i) mma_16816<F16>(d4, A[i].x, A[i].y, A[i].z, A[i].w, wb[gi][k][0], wb[gi][k][NE - 1]);
              o0[2 * k] = d4[0]; o0[2 * k + 1] = d4[1]; o1[2 * k] = d4[2]; o1[2 * k + 1] = d4[3];
            }
            uint32_t r0[4], r1[4];
            uint4 h0 = make_uint4(0u, 0u, 0u, 0u), h1 = h0;
            if (add) {
              h0 = *reinterpret_cast<const uint4*>(old + gi * 1024);
              h1 = *reinterpret_cast<const uint4*>(old + gi * 1024 + 512);
            }
            const uint32_t* q0 = reinterpret_cast<const uint32_t*>(&h0);
            const uint32_t* q1 = reinterpret_cast<const uint32_t*>(&h1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f0 = H::unpack(q0[i]), f1 = H::unpack(q1[i]);
              r0[i] = H::pack(fmaf(o0[2 * i], inv.row[0], f0.x), fmaf(o0[2 * i + 1], inv.row[0], f0.y));
              r1[i] = H::pack(fmaf(o1[2 * i], inv.row[1], f1.x), fmaf(o1[2 * i + 1], inv.row[1], f1.y));
            }
            if (v0) __stcs(reinterpret_cast<uint4*>(dx + (size_t)t0 * D + gi * 32), make_uint4(r0[0], r0[1], r0[2], r0[3]));
            if (v1) __stcs(reinterpret_cast<uint4*>(dx + (size_t)t1 * D + gi * 32), make_uint4(r1[0], r1[1], r1[2], r1[3]));
          }
        }
      }
      copy_old(j + held_blocks);                   // this block's have been used
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&dl_empty[r]));
    }
    cp_wait<0>();
    // this block's part of dWg: expert rows g (and g + 8), columns 8k + 2c, + 1 of each group
    float* part = a.partials + (size_t)blockIdx.x * E * D + 2 * c;
#pragma unroll
    for (int gi = 0; gi < kFuGroups; ++gi)
      if (g0 + gi < g1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* s4 = acc[gi][k];
          const int d = (g0 + gi) * 32 + 8 * k;
          if (NE == 1) {
            if (g < E) *reinterpret_cast<float2*>(part + (size_t)g * D + d) = make_float2(s4[0] + s4[2], s4[1] + s4[3]);
          } else {
            if (g < E) *reinterpret_cast<float2*>(part + (size_t)g * D + d) = make_float2(s4[0], s4[1]);
            if (g + 8 < E) *reinterpret_cast<float2*>(part + (size_t)(g + 8) * D + d) = make_float2(s4[2], s4[3]);
          }
        }
      }
  }
  // after a wait that ran out: no load may outlive the block
  __syncthreads();
  if (*abort_flag && tid == 0) {
    for (int st = 0; st < stages; ++st)
      if (loads[st]) mbar_wait(smem_u32(&full[st]), (loads[st] - 1) & 1, nullptr, nullptr, 425);
    mbar_wait(smem_u32(wbar), 0, nullptr, nullptr, 426);
  }
}

// ---------------------------------------------------------------- fp32
// x goes by L1, which keeps the gate weight that every token takes
__device__ __forceinline__ float4 ld_past_l1(const float* p) {
  float4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}
// FFMA throughout (a tensor core would round x).  One warp per TOK tokens: lane l holds columns
// 4l + 128 i of their rows and of Wg's.  TOK: one where the tokens do not fill the device, else as many
// share each read of Wg as registers hold: four with up to 8 experts (T = 32768, D = 1152, loss alone:
// 70 us, two: 84), two above (32 experts, T = 8192: 83 us, four: 145).
template <int EP, int TOK>
__global__ void __launch_bounds__(TOK == 2 ? 256 : 128) seq_scores_f32_kernel(SeqBalArgs a) {
  constexpr int NW = TOK == 2 ? 8 : 4;           // but for TOK = 1, 16 tokens a block
  __shared__ float db_s[NW][EP], loss_s[NW];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int D = a.D, E = a.E;
  const int tb = (blockIdx.x * NW + w) * TOK;
  launch_dependents();
  int t_lo, t_hi;
  live_rows(a, t_lo, t_hi);
  // the tokens' gate gradients, lane k holding slot k (at most 32 experts), on their way meanwhile
  int slots[TOK], sel[TOK];
  float gate[TOK];
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const bool in = a.dgate && tb + i < a.T;
    slots[i] = in ? slots_of(a, tb + i) : 0;
    sel[i] = in && lane < a.Kmax ? a.topk_idx[(size_t)(tb + i) * a.Kmax + lane] : -1;
    gate[i] = in && lane < a.Kmax ? a.dgate[(size_t)(tb + i) * a.Kmax + lane] : 0.f;
  }
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
      xv[i] = t < a.T ? ld_past_l1(x + (size_t)t * D + d) : zero;
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
  const float bias = lane < E && a.bias ? a.bias[lane] : 0.f;
  grid_dependency_wait();
  const float aux = a.aux_scale / (float)max(*a.live, 1);
  int2 tok[TOK];
  float C[TOK];
  float db = 0.f, loss_w = 0.f;
#pragma unroll
  for (int i = 0; i < TOK; ++i) tok[i] = tb + i >= t_lo && tb + i < t_hi ? a.tok[tb + i] : make_int2(-1, 0);
#pragma unroll
  for (int i = 0; i < TOK; ++i)
    C[i] = tok[i].x >= 0 && lane < E ? __int_as_float(tok[i].y) * (float)a.counts[(size_t)tok[i].x * E + lane] : 0.f;
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const int t = tb + i;
    const bool in = tok[i].x >= 0 || (a.all_gates && t < a.T);
    float mine = -INFINITY;
#pragma unroll
    for (int e = 0; e < EP; ++e)
      if (lane == e && e < E) mine = l[i][e] + bias;
    float m = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float pe = lane < E ? expf(mine - m) : 0.f;
    float z = pe;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float P = pe * (1.0f / z);
    float dp = aux * C[i];
    const int ns = in ? slots[i] : 0;              // the same in every lane
    for (int k = 0; k < ns; ++k) {
      const int e = __shfl_sync(0xffffffffu, sel[i], k);
      const float v = __shfl_sync(0xffffffffu, gate[i], k);
      if (e == lane) dp += v;
    }
    float share = P * C[i], pc = P * dp;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      share += __shfl_xor_sync(0xffffffffu, share, o);
      pc += __shfl_xor_sync(0xffffffffu, pc, o);
    }
    share = in ? share : 0.f;
    const float dl = in && lane < E ? P * (dp - pc) : 0.f;
    if (t < a.T) {
      if (lane == 0) a.tok_loss[t] = share;
      if (a.grads && lane < EP) a.dl[(size_t)t * EP + lane] = dl;
    }
    db += dl;
    loss_w += share;
  }
  if (TOK == 1) return;                            // few tokens: the finish kernel adds them one by one
  if (lane < EP) db_s[w][lane] = db;
  if (lane == 0) loss_s[w] = loss_w;
  __syncthreads();
  if (threadIdx.x < EP && a.grads) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) sum += db_s[k][threadIdx.x];
    a.db_part[(size_t)blockIdx.x * EP + threadIdx.x] = sum;
  }
  if (threadIdx.x == 0) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) sum += loss_s[k];
    a.blk_loss[blockIdx.x] = sum;
  }
}

constexpr int kF32Unit = 4;                        // ranges are a multiple of this many tokens
// One block per (128 columns, four ranges of tokens), a warp to a range: lane l owns four
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
  const int t_begin = max(range * a.blocks_per_range * kF32Unit, t_lo);
  const int t_end = min(min(a.T, t_hi), (range + 1) * a.blocks_per_range * kF32Unit);
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
        xv[u] = in ? ld_past_l1(x + (size_t)(tb + u) * D) : zero;
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
// db sums `db_rows` rows of ep values: dl's own rows (fp32, few tokens) or the kernels' sums over tokens.
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
    constexpr int kRound = 20;                     // 148 partial sums over 8 warps: all on their way at once
    float sum = 0.f;
    for (int k0 = w; k0 < a.groups; k0 += NW * kRound) {
      float r[kRound];
#pragma unroll
      for (int u = 0; u < kRound; ++u)
        r[u] = k0 + u * NW < a.groups ? __ldcg(a.partials + (size_t)(k0 + u * NW) * stride + i) : 0.f;
#pragma unroll
      for (int u = 0; u < kRound; u += 4) sum += (r[u] + r[u + 1]) + (r[u + 2] + r[u + 3]);
    }
    ws[w][lane] = sum;
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

// Launch K as a programmatic dependent of the kernel before.  Its limit of dynamic shared memory, MOST, is
// raised once on each device.
template <auto K, int MOST, typename... Q>
cudaError_t chained(int grid, int threads, int smem, cudaStream_t s, const Q&... args) {
  if (MOST > 32 * 1024) {                          // with what a kernel declares, above the default 48 KB
    static std::atomic<unsigned long long> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
      if ((e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST)) != cudaSuccess) return e;
      raised.fetch_or(bit, std::memory_order_relaxed);
    }
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
  return cudaLaunchKernelEx(&cfg, K, args...);
}

template <int NE, bool F16>
cudaError_t launch16(const SeqBalArgs& a, cudaStream_t s) {
  const int nblk = (a.T + 15) / 16;
  if constexpr (NE <= 2) {
    if (a.fused) {
      using P = Parts<NE, F16>;
      const bool add = a.dx && a.accumulate;
      const FusedPlan f = fused_plan(a.D, NE, P::A + P::T, add);
      return chained<seq_fused_kernel<NE, F16>, kFuMaxSmem>(a.groups, kFuThreads,
                     fused_smem(a.D, NE, P::A + P::T, f.stages, f.held).total, s, *a.tmap_x, a, f.stages, f.held);
    }
  }
  cudaError_t e = chained<seq_scores_kernel<NE, F16>, kScSmem>((nblk + kScWarps - 1) / kScWarps, kScWarps * 32, kScSmem, s, a);
  if (e != cudaSuccess || !a.grads) return e;
  return chained<seq_grads_kernel<NE, F16>, GradRing<NE, F16>::Smem>(a.D / 64 * a.groups, 128, GradRing<NE, F16>::Smem, s, a);
}
template <int EP>
cudaError_t launch32(const SeqBalArgs& a, cudaStream_t s) {
  cudaError_t e = a.T <= kSbF32Single ? chained<seq_scores_f32_kernel<EP, 1>, 0>((a.T + 3) / 4, 128, 0, s, a)
                                      : chained<seq_scores_f32_kernel<EP, EP == 8 ? 4 : 2>, 0>((a.T + 15) / 16, EP == 8 ? 128 : 256, 0, s, a);
  if (e != cudaSuccess || !a.grads) return e;
  return chained<seq_grads_f32_kernel<EP>, EP * 2048>((a.D + 127) / 128 * a.groups, 128, EP * 2048, s, a);
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

size_t seq_balance_scale_bytes(int E, int dtype) {
  return dtype != MOE_F16 ? 0 : (E <= 16 ? Parts<1, true>::V : Parts<4, true>::V) * 8 * sizeof(float4);
}

bool seq_balance_fused(int D, int E, int dtype) {
  if (dtype == MOE_F32 || E > 16 || D < kFuMinD || D / 32 > kFuCols * kFuGroups) return false;
  return fused_plan(D, E <= 8 ? 1 : 2, (int)(seq_balance_frag_bytes(E, dtype) / 512), true).stages >= 2;
}

void seq_balance_plan(int T, int D, int E, int dtype, int* groups, int* blocks_per_range) {
  if (seq_balance_fused(D, E, dtype)) {     // one block an SM, token blocks in turn
    const int nblk = (T + 15) / 16;
    *groups = nblk < kSbSms ? nblk : kSbSms;
    *blocks_per_range = 0;
    return;
  }
  const int slabs = dtype == MOE_F32 ? (D + 127) / 128 : D / 64, unit = dtype == MOE_F32 ? kF32Unit : 16;
  const int nblk = (T + unit - 1) / unit;
  int r = kSbSms * (E <= 16 ? 3 : 2) / slabs * 4;  // one wave of blocks, four ranges each
  if (r > nblk) r = nblk;
  if (r < 1) r = 1;
  *blocks_per_range = (nblk + r - 1) / r;
  const int ranges = *blocks_per_range > 0 ? (nblk + *blocks_per_range - 1) / *blocks_per_range : 0;
  *groups = (ranges + 3) / 4;
}

// one from each router warp of the one kernel, or from each 16 tokens of the two
int seq_balance_db_rows(int T, int D, int E, int dtype, int groups) {
  return seq_balance_fused(D, E, dtype) ? groups * kFuRouters : (T + 15) / 16;
}

cudaError_t launch_seq_balance(const SeqBalArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.T <= kOneTokens && (long long)a.n_seqs * a.E <= kOneCounts && a.n_seqs < kOffSmem) {
    seq_count_kernel<true><<<1, kOneThreads, 0, s>>>(a);
    e = cudaGetLastError();
  } else {
    const long long counts = (long long)a.n_seqs * a.E;
    const int clear = (int)(counts < 256 * kCountThreads ? (counts + kCountThreads - 1) / kCountThreads : 256);
    seq_clear_kernel<<<clear > 0 ? clear : 1, kCountThreads, 0, s>>>(a.counts, counts, a.live);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = chained<seq_count_kernel<false>, 0>((a.T + kCountThreads - 1) / kCountThreads, kCountThreads, 0, s, a);
  }
  if (e != cudaSuccess) return e;
  if (a.dtype == MOE_F32)
    e = a.E <= 8 ? launch32<8>(a, s) : a.E <= 16 ? launch32<16>(a, s) : launch32<32>(a, s);
  else
    e = a.dtype == MOE_F16 ? launch16_e<true>(a, s) : launch16_e<false>(a, s);
  if (e != cudaSuccess) return e;
  const int wg_blocks = a.dwg ? a.E * a.D / 32 : 0, db_blocks = a.dbias ? a.E : 0;
  const bool one = a.dtype == MOE_F32 && a.T <= kSbF32Single;   // db and the losses token by token
  const int db_rows = one ? a.T : seq_balance_db_rows(a.T, a.D, a.E, a.dtype, a.groups);
  return chained<seq_finish_kernel, 0>(wg_blocks + db_blocks + a.n_seqs + 1, kFinThreads, 0, s, a,
                 (const float*)(one ? a.dl : a.db_part), db_rows, seq_balance_ep(a.E), wg_blocks, db_blocks);
}

}  // namespace moe
