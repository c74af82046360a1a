// The optimizer's part of a training step, over many tensors in one launch: the
// gradient norm with its clip factor, and AdamW with moments in 32 or in 8 bits.
//
// AdamW of step t, g the gradient times the clip factor:
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// p is the fp32 master; its 16-bit copy (the weight the layer reads) and the
// weights' moving average are written in the same pass.  Every element is read
// and written once and nothing is shared between elements but the 8-bit scales,
// so the kernel is bound by memory: 28 bytes an element with fp32 gradients and
// moments, 16.06 with 8-bit moments, plus 2 for a copy and 8 for the average.
//
// 8-bit moments.  256 consecutive elements of a tensor share a fp32 scale, the
// largest magnitude over 448; a moment is an e4m3 code times it.  The second
// moment is kept as its root r = sqrt(v), which halves the range (in powers of
// two) that the codes have to span.  A code's neighbours are 6 to 12% away while
// one step moves v by 1 - b2 (0.1%), so rounding to the nearest code would leave
// v where it is for ever; codes are rounded up or down at random instead, up with
// the probability that makes the stored value right on average.  The 16 random
// bits for each moment are a hash of (seed, step, tensor, element): a call has no
// other state, and repeats bit for bit.  A root that is not zero keeps a code of 1
// (4.4e-6 of its block's largest) at least: were it rounded to zero while the same
// element's first moment is not, the next step would divide that by little more than eps
// (one gradient of 1 among others of 1e-6: moves of 500 lr, against 1.6 with the floor).
// The average of such roots is too large, and their elements' steps the shorter.
//
// A block is 256 threads on chunks of 2048 elements; a warp owns 256 elements of a
// chunk, eight consecutive ones in each lane, so that they are exactly one scale's and
// every fp32 stream moves in 32-byte vectors (two of 16 bytes where a tensor is aligned
// to no more).  With fp32 moments there is a block for every chunk: handed out in order
// they keep each stream's traffic within a narrow window of memory, which DRAM rewards
// (a probe that only moves these streams: 6.86 TB/s, against 6.05 from one wave of
// blocks that walk the chunks in strides and drift apart).  106 M parameters, clipped,
// with moving average and 16-bit copy: 673 us (norm included), 740 with one wave.  With
// 8-bit moments the arithmetic weighs as much, and what a block works out before its
// first chunk counts: one wave, 334 us; a block for every chunk 361 to 380, for every
// eight adjacent ones 389 (before roots had a floor; one wave is 336 since).
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kOptThreads = 256;
constexpr int kOptChunk = kOptThreads * 8;         // elements of a block's chunk
constexpr int kOptPerSm = 4;                       // resident blocks: 64 registers a thread
constexpr int kOptCountInside = 1184;              // blocks up to which they count the step themselves: 50,000 additions to
                                                   // one word cost 60 us, a kernel for it 2
constexpr int kScaleBlock = 256;                   // elements that share a scale
constexpr int kNormChunk = kOptThreads * 16;
constexpr int kOptSmall = 40, kOptLarge = 340;     // tensors a launch's parameters hold: under 4 KB, under 32 KB
constexpr int kNormSmall = 140, kNormLarge = 1100;
constexpr int kNormMaxBlocks = 2048;               // on every device: the sum's order is part of the result

// Tensor of a chunk: the first whose chunks end behind it.
__device__ __forceinline__ int find_tensor(const int* chunk_end, int n, int chunk) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (chunk < chunk_end[mid]) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// ---------------------------------------------------------------- vectors of eight elements
__device__ __forceinline__ void ld8(const float* p, bool wide, float* f) {
  if (wide) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "l"(p));
  } else {
    const float4 u = *reinterpret_cast<const float4*>(p), v = *(reinterpret_cast<const float4*>(p) + 1);
    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w; f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
  }
}
__device__ __forceinline__ void st8(float* p, bool wide, const float* f) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};"
                 :: "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]), "l"(p)
                 : "memory");
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(f[4], f[5], f[6], f[7]);
  }
}
__device__ __forceinline__ void ld8_grad(const void* g, int dtype, long long i, bool wide, float* f) {
  if (dtype == 0) {
    ld8(static_cast<const float*>(g) + i, wide, f);
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g) + i);
    if (dtype == 1) bf16x8_to_f32(v, f);
    else f16x8_to_f32(v, f);
  }
}
__device__ __forceinline__ float load1(const void* g, int dtype, long long i) {
  if (dtype == 0) return static_cast<const float*>(g)[i];
  if (dtype == 1) return __bfloat162float(static_cast<const __nv_bfloat16*>(g)[i]);
  return __half2float(static_cast<const __half*>(g)[i]);
}

// ---------------------------------------------------------------- gradient norm
template <int CAP>
struct NormParams {
  const void* g[CAP];
  long long n[CAP];
  int chunk_end[CAP];
  uint8_t dtype[CAP], wide[CAP];   // wide: 32-byte aligned
  int tensors, chunks;
  int part0, nparts;       // this launch's first partial; partials of all launches (last launch only)
  int last;
  double mult, max_norm;
  OptCtl* ctl;
  double* parts;
};

__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kOptThreads / 32; ++w) s += sh[w];
  __syncthreads();
  return s;
}

// Squares are formed and summed in fp64: no gradient over- or underflows the sum,
// so the sum is finite exactly when every gradient is.
template <int CAP>
__global__ void __launch_bounds__(kOptThreads) grad_norm_kernel(const __grid_constant__ NormParams<CAP> a) {
  __shared__ double sh[kOptThreads / 32];
  __shared__ int is_last;
  launch_dependents();                             // the step's kernel, if it comes next, is set up meanwhile
  double s = 0.0;
  for (int chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    const int k = find_tensor(a.chunk_end, a.tensors, chunk);
    const long long n = a.n[k];
    const long long base = (long long)(chunk - (k ? a.chunk_end[k - 1] : 0)) * kNormChunk;
    const void* g = a.g[k];
    const int dt = a.dtype[k];
    if (base + kNormChunk <= n) {
      float f[16];
#pragma unroll
      for (int u = 0; u < 2; ++u) ld8_grad(g, dt, base + u * (kOptThreads * 8) + threadIdx.x * 8, a.wide[k], f + 8 * u);
      double c[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
      for (int u = 0; u < 16; ++u) c[u & 3] = fma((double)f[u], (double)f[u], c[u & 3]);
      s += (c[0] + c[1]) + (c[2] + c[3]);
    } else {
      for (long long i = base + threadIdx.x; i < n; i += kOptThreads) {
        const double f = load1(g, dt, i);
        s = fma(f, f, s);
      }
    }
  }
  s = block_sum(s, sh);
  if (threadIdx.x == 0) {
    a.parts[a.part0 + blockIdx.x] = s;
    if (a.last) {
      __threadfence();
      is_last = atomicAdd(&a.ctl->norm_done, 1u) == gridDim.x - 1;
    }
  }
  if (!a.last) return;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  s = 0.0;                                         // the last block: every partial, in a fixed order
  for (int i = threadIdx.x; i < a.nparts; i += kOptThreads) s += __ldcg(a.parts + i);
  s = block_sum(s, sh);
  if (threadIdx.x == 0) {
    const double norm = a.mult * sqrt(s);
    const bool bad = !(norm <= 1.7976931348623157e308);
    const double clip = a.max_norm > 0.0 ? fmin(1.0, a.max_norm / (norm + 1e-6)) : 1.0;
    a.ctl->grad_norm = (float)norm;
    a.ctl->grad_scale = bad ? 0.f : (float)(a.mult * clip);
    a.ctl->nonfinite = bad ? 1 : 0;
    a.ctl->norm_done = 0;
  }
}

// ---------------------------------------------------------------- AdamW
struct OptTensor {
  float* p; const void* g; void* w;
  void* m; void* v; float* ms; float* vs;
  float* ema;
  long long n;
  float wd;
  int index;               // place in the call's list: keys the rounding
  uint8_t gdt, wdt;
  uint8_t wide;            // every fp32 stream is 32-byte aligned
};
template <int CAP>
struct AdamwParams {
  OptTensor t[CAP];
  int chunk_end[CAP];
  int tensors, chunks;
  int clipped, last;       // last: 1 or 2 for the call's last launch; 2: its blocks count the step
  double lr, beta1, beta2, eps, ema_decay, mult;
  unsigned long long seed;
  OptCtl* ctl;
};

__device__ __forceinline__ void count_step(OptCtl& c, bool skip, double beta1, double beta2) {
  if (skip) {
    c.skipped += 1;
  } else {
    c.step += 1;
    c.beta1_t *= beta1;
    c.beta2_t *= beta2;
  }
}
__global__ void adamw_count_kernel(OptCtl* c, int clipped, double beta1, double beta2) {
  count_step(*c, clipped && c->nonfinite, beta1, beta2);
}

// One step's scalars.
struct StepScalars {
  float scale, b1, omb1, b2, omb2, step_size, rs2, eps, ed, omed;
  double lr;
  int skip;
  long long t;
};

// 64-bit key of a step's k-th tensor.  The odd multipliers are the fractions of 1/phi and of the
// square roots of 3 and 2.
__device__ __forceinline__ unsigned long long tensor_key(unsigned long long seed, long long step, int k) {
  unsigned long long h = seed + (unsigned long long)step * 0x9E3779B97F4A7C15ull +
                         (unsigned long long)k * 0xBB67AE8584CAA73Bull;
  h = (h ^ (h >> 29)) * 0x6A09E667F3BCC909ull;
  return (h ^ (h >> 32)) >> 1;
}
// 32 random bits for an element: twice a 32 x 32 -> 64 bit product, folded.
__device__ __forceinline__ uint32_t element_bits(uint32_t i_plus_key_lo, uint32_t key_hi) {
  unsigned long long z = (unsigned long long)i_plus_key_lo * 0x9E3779B9u;
  z = (unsigned long long)((uint32_t)z ^ (uint32_t)(z >> 32) ^ key_hi) * 0x6A09E667u;
  return (uint32_t)z ^ (uint32_t)(z >> 32);
}

// |x| <= 448 (a rounding or two above) to the code of a neighbouring e4m3 value, in the top byte.
// Times 2^-120 the e4m3 exponents are fp32's own and e4m3's subnormals fp32's, so that bits 26..20
// are the code of the value below in magnitude.  16 random bits under them carry with the probability
// that the rest is worth, into subnormals and binades alike; their own four zero bits below leave
// room for a rounding above 448.
__device__ __forceinline__ uint32_t e4m3_random(float x, uint32_t r16_shl8) {
  return (__float_as_uint(__fmul_rn(x, 0x1p-120f)) << 4) + r16_shl8;   // the sign is shifted out
}
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}
__device__ __forceinline__ float2 e4m3_values(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(__half2(h));
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// m, v and the root in the roundings of their formulas written out (no contraction, IEEE square
// root): what is kept does not depend on how a compiler fuses them.  The update's quotient goes
// through an approximate reciprocal (one unit in the last place): it is then scaled by lr and added
// to a parameter some thousand times larger.  A denominator below 2^-70 counts as that: the square of a
// gradient below 8.4e-22, about 2^-70, times 1 - b2 = 0.001 is zero in fp32 (a root that is not is 2^-75 at
// least), and with eps = 0 its first moment, which is not, would be divided by nothing.
__device__ __forceinline__ float moments(float g, float& m, float& v, const StepScalars& s) {
  m = __fadd_rn(__fmul_rn(s.b1, m), __fmul_rn(s.omb1, g));
  v = __fadd_rn(__fmul_rn(s.b2, v), __fmul_rn(s.omb2, __fmul_rn(g, g)));
  return __fsqrt_rn(v);
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float update(float p, float m, float root, float keep, const StepScalars& s) {
  const float den = max_nan(fmaf(root, s.rs2, s.eps), 0x1p-70f);
  return fmaf(-s.step_size, m * rcp_approx(den), __fmul_rn(p, keep));
}

template <bool Q8, int CAP>
__global__ void __launch_bounds__(kOptThreads, kOptPerSm) adamw_kernel(const __grid_constant__ AdamwParams<CAP> a) {
  __shared__ StepScalars ss;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();                          // a programmatic dependent of what runs before (the norm)
  if (tid == 0) {
    const OptCtl& c = *a.ctl;
    const double c1 = 1.0 - c.beta1_t * a.beta1, c2 = 1.0 - c.beta2_t * a.beta2;
    ss.lr = a.lr * (double)c.lr_scale;
    ss.scale = a.clipped ? c.grad_scale : (float)a.mult;
    ss.b1 = (float)a.beta1; ss.omb1 = (float)(1.0 - a.beta1);
    ss.b2 = (float)a.beta2; ss.omb2 = (float)(1.0 - a.beta2);
    ss.step_size = (float)(ss.lr / c1);
    ss.rs2 = (float)(1.0 / sqrt(c2));
    ss.eps = (float)a.eps;
    ss.ed = (float)a.ema_decay; ss.omed = (float)(1.0 - a.ema_decay);
    ss.skip = a.clipped && c.nonfinite;
    ss.t = c.step + 1;
  }
  __syncthreads();
  const StepScalars s = ss;
  if (!s.skip) {
    // From the last chunk to the first: the norm's pass has left the last gradients in L2.  What belongs to
    // a tensor is worked out when its first chunk comes.
    int k = a.tensors, first = a.chunks;           // the current tensor and its first chunk
    long long n = 0;
    float keep = 0.f;
    uint32_t key_lo = 0, key_hi = 0;
    for (int chunk = a.chunks - 1 - (int)blockIdx.x; chunk >= 0; chunk -= (int)gridDim.x) {
      if (chunk < first) {
        k = find_tensor(a.chunk_end, k, chunk);
        first = k ? a.chunk_end[k - 1] : 0;
        n = a.t[k].n;
        keep = (float)(1.0 - s.lr * (double)a.t[k].wd);
        if (Q8) {
          const unsigned long long key = tensor_key(a.seed, s.t, a.t[k].index);
          key_lo = (uint32_t)key;
          key_hi = (uint32_t)(key >> 32);
        }
      }
      const OptTensor& t = a.t[k];
      const long long wbase = (long long)(chunk - first) * kOptChunk + warp * kScaleBlock;
      if (wbase >= n) continue;
      const bool full = wbase + kScaleBlock <= n, wide = t.wide;
      const long long i0 = wbase + lane * 8;
      const long long sb = wbase / kScaleBlock;
      float* const tm = static_cast<float*>(t.m);
      float* const tv = static_cast<float*>(t.v);
      uint8_t* const qm = static_cast<uint8_t*>(t.m);
      uint8_t* const qv = static_cast<uint8_t*>(t.v);
      float g[8], p[8], m[8], v[8], e[8], r[8];
      uint2 mc = make_uint2(0u, 0u), vc = mc;
      float ms = 0.f, vs = 0.f;
      if (Q8) {
        ms = t.ms[sb];
        vs = t.vs[sb];
      }
      if (full) {
        ld8_grad(t.g, t.gdt, i0, wide, g);
        ld8(t.p + i0, wide, p);
        if (Q8) {
          mc = *reinterpret_cast<const uint2*>(qm + i0);
          vc = *reinterpret_cast<const uint2*>(qv + i0);
        } else {
          ld8(tm + i0, wide, m);
          ld8(tv + i0, wide, v);
        }
        if (t.ema) ld8(t.ema + i0, wide, e);
      } else {                                     // the tensor's end: zeros past it, which stay zero
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const bool in = i0 + q < n;
          g[q] = in ? load1(t.g, t.gdt, i0 + q) : 0.f;
          p[q] = in ? t.p[i0 + q] : 0.f;
          if (Q8) {
            if (in) {
              (q < 4 ? mc.x : mc.y) |= (uint32_t)qm[i0 + q] << (8 * (q & 3));
              (q < 4 ? vc.x : vc.y) |= (uint32_t)qv[i0 + q] << (8 * (q & 3));
            }
          } else {
            m[q] = in ? tm[i0 + q] : 0.f;
            v[q] = in ? tv[i0 + q] : 0.f;
          }
          e[q] = in && t.ema ? t.ema[i0 + q] : 0.f;
        }
      }
      if (Q8) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float2 a2 = e4m3_values((h < 2 ? mc.x : mc.y) >> (16 * (h & 1)) & 0xffffu);
          const float2 b2 = e4m3_values((h < 2 ? vc.x : vc.y) >> (16 * (h & 1)) & 0xffffu);
          m[2 * h] = __fmul_rn(a2.x, ms); m[2 * h + 1] = __fmul_rn(a2.y, ms);
          v[2 * h] = __fmul_rn(b2.x, vs); v[2 * h + 1] = __fmul_rn(b2.y, vs);
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (Q8) v[q] = __fmul_rn(v[q], v[q]);      // what is stored is the root
        r[q] = moments(__fmul_rn(g[q], s.scale), m[q], v[q], s);
        p[q] = update(p[q], m[q], r[q], keep, s);
      }
      if (Q8) {
        float mx = 0.f, vx = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          mx = max_nan(mx, fabsf(m[q]));
          vx = max_nan(vx, r[q]);
        }
        // non-negative floats order as their bits do, and a NaN lies above them
        const uint32_t um = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
        const uint32_t uv = __reduce_max_sync(0xffffffffu, __float_as_uint(vx));
        mx = __uint_as_float(um);
        vx = __uint_as_float(uv);
        // a block whose largest moment is below 2^-100, or not finite, becomes zero; first moments also where the
        // second are not finite (gradients from 1.8e19 on): they would be divided by the next gradient alone.
        // One unsigned comparison holds both ends of a range.
        constexpr uint32_t kLow = 0x0d800000u, kInf = 0x7f800000u;
        const bool mok = um - kLow < kInf - kLow && uv < kInf, vok = uv - kLow < kInf - kLow;
        const float mi = mok ? __fmul_rn(__frcp_rn(mx), 448.f) : 0.f, vi = vok ? __fmul_rn(__frcp_rn(vx), 448.f) : 0.f;
        const uint32_t klo = key_lo + (uint32_t)i0;
        if (!mok) {
#pragma unroll
          for (int q = 0; q < 8; ++q) m[q] = 0.f;
        }
        if (!vok) {
#pragma unroll
          for (int q = 0; q < 8; ++q) r[q] = 0.f;
        }
        uint32_t zm[8], zv[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t rnd = element_bits(klo + q, key_hi);
          zm[q] = e4m3_random(__fmul_rn(m[q], mi), __byte_perm(rnd, 0u, 0x4104)) | (__float_as_uint(m[q]) & 0x80000000u);
          zv[q] = e4m3_random(__fmul_rn(r[q], vi), __byte_perm(rnd, 0u, 0x4324));
        }
        mc = make_uint2(top_bytes(zm[0], zm[1], zm[2], zm[3]), top_bytes(zm[4], zm[5], zm[6], zm[7]));
        vc = make_uint2(top_bytes(zv[0], zv[1], zv[2], zv[3]), top_bytes(zv[4], zv[5], zv[6], zv[7]));
        // a code (below 128) plus 127 has its top bit set unless it is 0: rarely one is, and only then each root is
        // looked at (106 M parameters, back to back: 336 us, with a maximum for every code 343, unguarded 332)
        if (((vc.x + 0x7f7f7f7fu) & (vc.y + 0x7f7f7f7fu) & 0x80808080u) != 0x80808080u) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (r[q] > 0.f) zv[q] = max(zv[q], 0x01000000u);
          vc = make_uint2(top_bytes(zv[0], zv[1], zv[2], zv[3]), top_bytes(zv[4], zv[5], zv[6], zv[7]));
        }
        if (lane == 0) {
          t.ms[sb] = mok ? __fmul_rn(mx, 1.f / 448.f) : 0.f;
          t.vs[sb] = vok ? __fmul_rn(vx, 1.f / 448.f) : 0.f;
        }
      }
      if (full) {
        st8(t.p + i0, wide, p);
        if (Q8) {
          *reinterpret_cast<uint2*>(qm + i0) = mc;
          *reinterpret_cast<uint2*>(qv + i0) = vc;
        } else {
          st8(tm + i0, wide, m);
          st8(tv + i0, wide, v);
        }
        if (t.ema) {
#pragma unroll
          for (int q = 0; q < 8; ++q) e[q] = __fadd_rn(__fmul_rn(s.ed, e[q]), __fmul_rn(s.omed, p[q]));
          st8(t.ema + i0, wide, e);
        }
        if (t.w) {                                 // the next forward reads it: left in L2
          const uint4 w = t.wdt == 1 ? make_uint4(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]),
                                                  pack_bf16x2(p[4], p[5]), pack_bf16x2(p[6], p[7]))
                                     : make_uint4(pack_f16x2(p[0], p[1]), pack_f16x2(p[2], p[3]),
                                                  pack_f16x2(p[4], p[5]), pack_f16x2(p[6], p[7]));
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(t.w) + i0) = w;
        }
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const long long i = i0 + q;
          if (i >= n) continue;
          t.p[i] = p[q];
          if (Q8) {
            qm[i] = (uint8_t)((q < 4 ? mc.x : mc.y) >> (8 * (q & 3)));
            qv[i] = (uint8_t)((q < 4 ? vc.x : vc.y) >> (8 * (q & 3)));
          } else {
            tm[i] = m[q];
            tv[i] = v[q];
          }
          if (t.ema) t.ema[i] = __fadd_rn(__fmul_rn(s.ed, e[q]), __fmul_rn(s.omed, p[q]));
          if (t.w && t.wdt == 1) static_cast<__nv_bfloat16*>(t.w)[i] = __float2bfloat16_rn(p[q]);
          else if (t.w) static_cast<__half*>(t.w)[i] = __float2half_rn(p[q]);
        }
      }
    }
  }
  // the last block of the call's last launch counts the step: every block has read the control block
  if (a.last == 2 && tid == 0) {
    __threadfence();
    if (atomicAdd(&a.ctl->step_done, 1u) == gridDim.x - 1) {
      count_step(*a.ctl, s.skip, a.beta1, a.beta2);
      a.ctl->step_done = 0;
    }
  }
}

__global__ void optim_init_kernel(OptCtl* c, long long step, double b1t, double b2t) {
  OptCtl v{};
  v.step = step;
  v.beta1_t = b1t;
  v.beta2_t = b2t;
  v.lr_scale = 1.f;
  v.grad_scale = 1.f;
  *c = v;
}

template <int CAP>
cudaError_t norm_launch(const moe_adamw_tensor_t* t, int n, double mult, double max_norm, OptCtl* ctl, double* parts,
                        int* part0, bool last, cudaStream_t s) {
  static_assert(sizeof(NormParams<CAP>) <= 32764, "kernel parameters");
  NormParams<CAP> a;
  long long chunks = 0;
  a.tensors = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].n == 0) continue;
    chunks += (t[i].n + kNormChunk - 1) / kNormChunk;
    a.g[a.tensors] = t[i].grad;
    a.n[a.tensors] = t[i].n;
    a.dtype[a.tensors] = (uint8_t)t[i].grad_dtype;
    a.wide[a.tensors] = ((uintptr_t)t[i].grad & 31u) == 0;
    a.chunk_end[a.tensors++] = (int)chunks;
  }
  a.chunks = (int)chunks;
  a.part0 = *part0;
  a.last = last;
  a.mult = mult; a.max_norm = max_norm; a.ctl = ctl; a.parts = parts;
  const int grid = (int)(chunks < 1 ? 1 : chunks < kNormMaxBlocks ? chunks : kNormMaxBlocks);
  *part0 += grid;
  a.nparts = *part0;
  grad_norm_kernel<CAP><<<grid, kOptThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <bool Q8, int CAP>
cudaError_t adamw_launch(const moe_adamw_t& h, const moe_adamw_tensor_t* t, int first, int n, OptCtl* ctl, bool last,
                         int sms, cudaStream_t s) {
  static_assert(sizeof(AdamwParams<CAP>) <= 32764, "kernel parameters");
  AdamwParams<CAP> a;
  long long chunks = 0;
  a.tensors = 0;
  for (int i = first; i < first + n; ++i) {
    if (t[i].n == 0) continue;
    chunks += (t[i].n + kOptChunk - 1) / kOptChunk;
    OptTensor& o = a.t[a.tensors];
    o.p = t[i].param; o.g = t[i].grad; o.w = t[i].weight;
    o.m = t[i].m; o.v = t[i].v; o.ms = t[i].m_scale; o.vs = t[i].v_scale;
    o.ema = t[i].ema;
    o.n = t[i].n; o.wd = t[i].weight_decay; o.index = i;
    o.gdt = (uint8_t)t[i].grad_dtype; o.wdt = (uint8_t)t[i].weight_dtype;
    uintptr_t at = (uintptr_t)o.p | (uintptr_t)o.ema;
    if (o.gdt == MOE_F32) at |= (uintptr_t)o.g;
    if (!Q8) at |= (uintptr_t)o.m | (uintptr_t)o.v;
    o.wide = (at & 31u) == 0;
    a.chunk_end[a.tensors++] = (int)chunks;
  }
  a.chunks = (int)chunks;
  a.clipped = h.clipped;
  a.lr = h.lr; a.beta1 = h.beta1; a.beta2 = h.beta2; a.eps = h.eps; a.ema_decay = h.ema_decay; a.mult = h.grad_mult;
  a.seed = h.seed;
  a.ctl = ctl;
  const long long wave = (long long)sms * kOptPerSm;
  const int grid = (int)(chunks < 1 ? 1 : Q8 && chunks > wave ? wave : chunks);
  a.last = !last ? 0 : grid <= kOptCountInside ? 2 : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kOptThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, adamw_kernel<Q8, CAP>, a);
  if (e != cudaSuccess || a.last != 1) return e;
  adamw_count_kernel<<<1, 1, 0, s>>>(ctl, h.clipped, h.beta1, h.beta2);
  return cudaGetLastError();
}

template <bool Q8>
cudaError_t adamw_all(const moe_adamw_t& h, const moe_adamw_tensor_t* t, int n, OptCtl* ctl, int sms, cudaStream_t s) {
  if (n <= kOptSmall) return adamw_launch<Q8, kOptSmall>(h, t, 0, n, ctl, true, sms, s);
  for (int first = 0; first < n; first += kOptLarge) {
    const int k = n - first < kOptLarge ? n - first : kOptLarge;
    const cudaError_t e = adamw_launch<Q8, kOptLarge>(h, t, first, k, ctl, first + k == n, sms, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_norm_scratch(int n) {
  const size_t launches = n <= kNormSmall ? 1 : (size_t)(n + kNormLarge - 1) / kNormLarge;
  return launches * kNormMaxBlocks * sizeof(double);
}

cudaError_t launch_optim_init(OptCtl* c, long long step, double b1t, double b2t, cudaStream_t s) {
  optim_init_kernel<<<1, 1, 0, s>>>(c, step, b1t, b2t);
  return cudaGetLastError();
}

cudaError_t launch_grad_norm(const moe_adamw_tensor_t* t, int n, double mult, double max_norm, OptCtl* ctl, double* parts,
                             cudaStream_t s) {
  int part0 = 0;
  if (n <= kNormSmall) return norm_launch<kNormSmall>(t, n, mult, max_norm, ctl, parts, &part0, true, s);
  for (int first = 0; first < n; first += kNormLarge) {
    const int k = n - first < kNormLarge ? n - first : kNormLarge;
    const cudaError_t e =
        norm_launch<kNormLarge>(t + first, k, mult, max_norm, ctl, parts, &part0, first + k == n, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_adamw(const moe_adamw_t& h, const moe_adamw_tensor_t* t, int n, OptCtl* ctl, int sms, cudaStream_t s) {
  return h.state == MOE_MOMENTS_E4M3 ? adamw_all<true>(h, t, n, ctl, sms, s) : adamw_all<false>(h, t, n, ctl, sms, s);
}

}  // namespace moe
