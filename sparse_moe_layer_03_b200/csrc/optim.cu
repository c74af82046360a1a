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
// other state, and repeats bit for bit.
//
// One block is 256 threads on a chunk of 2048 elements; a warp owns 256 of them,
// four consecutive ones in each lane and then four again 128 further on, so that
// every 32-bit stream moves in 512-byte pieces and a warp's elements are exactly
// one scale's.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kOptThreads = 256;
constexpr int kOptChunk = kOptThreads * 8;         // elements of a block's chunk
constexpr int kScaleBlock = 256;                   // elements that share a scale
constexpr int kNormChunk = kOptThreads * 16;
constexpr int kOptSmall = 40, kOptLarge = 340;     // tensors a launch's parameters hold: under 4 KB, under 32 KB
constexpr int kNormSmall = 140, kNormLarge = 1100;
constexpr int kNormMaxBlocks = 2048;

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

// ---------------------------------------------------------------- gradient loads
__device__ __forceinline__ void load4(const void* g, int dtype, long long i, float* f) {
  if (dtype == 0) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(g) + i));
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g) + i));
    if (dtype == 1) {
      f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
      f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
    } else {
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
      f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    }
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
  uint8_t dtype[CAP];
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
      for (int u = 0; u < 4; ++u) load4(g, dt, base + u * (kOptThreads * 4) + threadIdx.x * 4, f + 4 * u);
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
};
template <int CAP>
struct AdamwParams {
  OptTensor t[CAP];
  int chunk_end[CAP];
  int tensors, chunks;
  int clipped, last;
  double lr, beta1, beta2, eps, ema_decay, mult;
  unsigned long long seed;
  OptCtl* ctl;
};

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
__device__ __forceinline__ uint32_t element_bits(uint32_t i, uint32_t key_lo, uint32_t key_hi) {
  unsigned long long z = (unsigned long long)(i + key_lo) * 0x9E3779B9u;
  z = (unsigned long long)((uint32_t)z ^ (uint32_t)(z >> 32) ^ key_hi) * 0x6A09E667u;
  return (uint32_t)z ^ (uint32_t)(z >> 32);
}

// |x| <= 448 (a rounding above) to an e4m3 code: the fp32 bits below the code's three mantissa bits,
// plus 16 random ones at their top, carry into the code with the probability that they are worth.
// Below 2^-6 the codes are 2^-9 apart: adding 2^-6 gives the value that spacing.
__device__ __forceinline__ uint32_t e4m3_code(float x, uint32_t r16) {
  const float a = fabsf(x);
  const bool low = a < 0.015625f;
  const uint32_t bits = __float_as_uint(low ? a + 0.015625f : a) + (r16 << 4);
  int code = (int)(bits >> 20) - (low ? 968 : 960);
  code = code < 126 ? code : 126;
  return (uint32_t)code | (x < 0.f ? 128u : 0u);
}
// an e4m3 code's value: its exponent and mantissa moved to fp16's place (8 below in exponent), exactly
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const uint16_t h = (uint16_t)(((code & 0x80u) << 8) | ((code & 0x7fu) << 7));
  return __half2float(__ushort_as_half(h)) * 256.f;
}

// m, v and the update in the same roundings as their formulas written out (no contraction), so that
// the moments do not depend on how a compiler fuses them.  The update's quotient may be off by two
// units: it is then scaled by lr and added to a parameter some thousand times larger.
__device__ __forceinline__ float moments(float g, float& m, float& v, const StepScalars& s) {
  m = __fadd_rn(__fmul_rn(s.b1, m), __fmul_rn(s.omb1, g));
  v = __fadd_rn(__fmul_rn(s.b2, v), __fmul_rn(s.omb2, __fmul_rn(g, g)));
  return __fsqrt_rn(v);
}
__device__ __forceinline__ float update(float p, float m, float root, float keep, const StepScalars& s) {
  return fmaf(-s.step_size, __fdividef(m, fmaf(root, s.rs2, s.eps)), __fmul_rn(p, keep));
}

template <bool Q8, int CAP>
__global__ void __launch_bounds__(kOptThreads) adamw_kernel(const __grid_constant__ AdamwParams<CAP> a) {
  __shared__ StepScalars ss;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    for (int chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
      const int k = find_tensor(a.chunk_end, a.tensors, chunk);
      const OptTensor& t = a.t[k];
      const long long n = t.n;
      const long long wbase = (long long)(chunk - (k ? a.chunk_end[k - 1] : 0)) * kOptChunk + warp * kScaleBlock;
      if (wbase >= n) continue;
      const float keep = (float)(1.0 - s.lr * (double)t.wd);
      float g[8], p[8], m[8], v[8], e[8];
      const bool full = wbase + kScaleBlock <= n;
      const float ms = Q8 ? t.ms[wbase / kScaleBlock] : 0.f, vs = Q8 ? t.vs[wbase / kScaleBlock] : 0.f;
      if (full) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const long long i = wbase + u * 128 + lane * 4;
          load4(t.g, t.gdt, i, g + 4 * u);
          const float4 pv = __ldcs(reinterpret_cast<const float4*>(t.p + i));
          p[4 * u] = pv.x; p[4 * u + 1] = pv.y; p[4 * u + 2] = pv.z; p[4 * u + 3] = pv.w;
          if (Q8) {
            const uint32_t mc = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + i));
            const uint32_t vc = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + i));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              m[4 * u + q] = __fmul_rn(e4m3_value((mc >> (8 * q)) & 255u), ms);
              v[4 * u + q] = __fmul_rn(e4m3_value((vc >> (8 * q)) & 255u), vs);
            }
          } else {
            const float4 mv = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(t.m) + i));
            const float4 vv = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(t.v) + i));
            m[4 * u] = mv.x; m[4 * u + 1] = mv.y; m[4 * u + 2] = mv.z; m[4 * u + 3] = mv.w;
            v[4 * u] = vv.x; v[4 * u + 1] = vv.y; v[4 * u + 2] = vv.z; v[4 * u + 3] = vv.w;
          }
          if (t.ema) {
            const float4 ev = __ldcs(reinterpret_cast<const float4*>(t.ema + i));
            e[4 * u] = ev.x; e[4 * u + 1] = ev.y; e[4 * u + 2] = ev.z; e[4 * u + 3] = ev.w;
          }
        }
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {              // the tensor's end: zeros past it, which stay zero
          const long long i = wbase + (q >> 2) * 128 + lane * 4 + (q & 3);
          const bool in = i < n;
          g[q] = in ? load1(t.g, t.gdt, i) : 0.f;
          p[q] = in ? t.p[i] : 0.f;
          if (Q8) {
            m[q] = in ? __fmul_rn(e4m3_value(static_cast<const uint8_t*>(t.m)[i]), ms) : 0.f;
            v[q] = in ? __fmul_rn(e4m3_value(static_cast<const uint8_t*>(t.v)[i]), vs) : 0.f;
          } else {
            m[q] = in ? static_cast<const float*>(t.m)[i] : 0.f;
            v[q] = in ? static_cast<const float*>(t.v)[i] : 0.f;
          }
          e[q] = in && t.ema ? t.ema[i] : 0.f;
        }
      }
      float r[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (Q8) v[q] = __fmul_rn(v[q], v[q]);      // what is stored is the root
        r[q] = moments(__fmul_rn(g[q], s.scale), m[q], v[q], s);
        p[q] = update(p[q], m[q], r[q], keep, s);
        e[q] = t.ema ? __fadd_rn(__fmul_rn(s.ed, e[q]), __fmul_rn(s.omed, p[q])) : 0.f;
      }
      uint32_t mc[8], vc[8];
      if (Q8) {
        uint32_t mb = 0, vb = 0;                   // non-negative floats order as their bits do
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          mb = max(mb, __float_as_uint(fabsf(m[q])));
          vb = max(vb, __float_as_uint(r[q]));
        }
        const float mx = __uint_as_float(__reduce_max_sync(0xffffffffu, mb));
        const float vx = __uint_as_float(__reduce_max_sync(0xffffffffu, vb));
        // a block whose largest moment is below 2^-100, or not finite, becomes zero
        const bool mok = mx >= 7.888609052210118e-31f && mx < INFINITY, vok = vx >= 7.888609052210118e-31f && vx < INFINITY;
        const float mi = mok ? __fdiv_rn(448.f, mx) : 0.f, vi = vok ? __fdiv_rn(448.f, vx) : 0.f;
        const unsigned long long key = tensor_key(a.seed, s.t, t.index);
        const uint32_t klo = (uint32_t)key, khi = (uint32_t)(key >> 32);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t rnd = element_bits((uint32_t)(wbase + (q >> 2) * 128 + lane * 4 + (q & 3)), klo, khi);
          mc[q] = e4m3_code(__fmul_rn(m[q], mi), rnd & 0xffffu);
          vc[q] = e4m3_code(__fmul_rn(r[q], vi), rnd >> 16);
        }
        if (lane == 0) {
          t.ms[wbase / kScaleBlock] = mok ? __fdiv_rn(mx, 448.f) : 0.f;
          t.vs[wbase / kScaleBlock] = vok ? __fdiv_rn(vx, 448.f) : 0.f;
        }
      }
      if (full) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const long long i = wbase + u * 128 + lane * 4;
          __stcs(reinterpret_cast<float4*>(t.p + i), make_float4(p[4 * u], p[4 * u + 1], p[4 * u + 2], p[4 * u + 3]));
          if (Q8) {
            uint32_t mw = 0, vw = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              mw |= mc[4 * u + q] << (8 * q);
              vw |= vc[4 * u + q] << (8 * q);
            }
            __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + i), mw);
            __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + i), vw);
          } else {
            __stcs(reinterpret_cast<float4*>(static_cast<float*>(t.m) + i),
                   make_float4(m[4 * u], m[4 * u + 1], m[4 * u + 2], m[4 * u + 3]));
            __stcs(reinterpret_cast<float4*>(static_cast<float*>(t.v) + i),
                   make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]));
          }
          if (t.ema)
            __stcs(reinterpret_cast<float4*>(t.ema + i), make_float4(e[4 * u], e[4 * u + 1], e[4 * u + 2], e[4 * u + 3]));
          if (t.w) {
            const uint2 w = t.wdt == 1 ? make_uint2(pack_bf16x2(p[4 * u], p[4 * u + 1]), pack_bf16x2(p[4 * u + 2], p[4 * u + 3]))
                                       : make_uint2(pack_f16x2(p[4 * u], p[4 * u + 1]), pack_f16x2(p[4 * u + 2], p[4 * u + 3]));
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(t.w) + i) = w;   // the next forward reads it: kept in L2
          }
        }
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const long long i = wbase + (q >> 2) * 128 + lane * 4 + (q & 3);
          if (i >= n) continue;
          t.p[i] = p[q];
          if (Q8) {
            static_cast<uint8_t*>(t.m)[i] = (uint8_t)mc[q];
            static_cast<uint8_t*>(t.v)[i] = (uint8_t)vc[q];
          } else {
            static_cast<float*>(t.m)[i] = m[q];
            static_cast<float*>(t.v)[i] = v[q];
          }
          if (t.ema) t.ema[i] = e[q];
          if (t.w && t.wdt == 1) static_cast<__nv_bfloat16*>(t.w)[i] = __float2bfloat16_rn(p[q]);
          else if (t.w) static_cast<__half*>(t.w)[i] = __float2half_rn(p[q]);
        }
      }
    }
  }
  // the last block of the call's last launch counts the step: every block has read the control block
  if (a.last && tid == 0) {
    __threadfence();
    if (atomicAdd(&a.ctl->step_done, 1u) == gridDim.x - 1) {
      OptCtl& c = *a.ctl;
      if (s.skip) {
        c.skipped += 1;
      } else {
        c.step = s.t;
        c.beta1_t *= a.beta1;
        c.beta2_t *= a.beta2;
      }
      c.step_done = 0;
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
                        int* part0, bool last, int blocks_max, cudaStream_t s) {
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
    a.chunk_end[a.tensors++] = (int)chunks;
  }
  a.chunks = (int)chunks;
  a.part0 = *part0;
  a.last = last;
  a.mult = mult; a.max_norm = max_norm; a.ctl = ctl; a.parts = parts;
  const int grid = (int)(chunks < 1 ? 1 : chunks < blocks_max ? chunks : blocks_max);
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
    a.chunk_end[a.tensors++] = (int)chunks;
  }
  a.chunks = (int)chunks;
  a.clipped = h.clipped; a.last = last;
  a.lr = h.lr; a.beta1 = h.beta1; a.beta2 = h.beta2; a.eps = h.eps; a.ema_decay = h.ema_decay; a.mult = h.grad_mult;
  a.seed = h.seed;
  a.ctl = ctl;
  const long long most = (long long)sms * 4;
  const int grid = (int)(chunks < 1 ? 1 : chunks < most ? chunks : most);
  adamw_kernel<Q8, CAP><<<grid, kOptThreads, 0, s>>>(a);
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
                             int sms, cudaStream_t s) {
  int part0 = 0;
  const int most = sms * 8 < kNormMaxBlocks ? sms * 8 : kNormMaxBlocks;
  if (n <= kNormSmall) return norm_launch<kNormSmall>(t, n, mult, max_norm, ctl, parts, &part0, true, most, s);
  for (int first = 0; first < n; first += kNormLarge) {
    const int k = n - first < kNormLarge ? n - first : kNormLarge;
    const cudaError_t e =
        norm_launch<kNormLarge>(t + first, k, mult, max_norm, ctl, parts, &part0, first + k == n, most, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_adamw(const moe_adamw_t& h, const moe_adamw_tensor_t* t, int n, OptCtl* ctl, int sms, cudaStream_t s) {
  return h.state == MOE_MOMENTS_E4M3 ? adamw_all<true>(h, t, n, ctl, sms, s) : adamw_all<false>(h, t, n, ctl, sms, s);
}

}  // namespace moe
