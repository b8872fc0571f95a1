// optim.cu — the global gradient norm and the AdamW step over many tensors.
//
// Both walk a list of tensors in one launch: the list is cut into blocks of
// 256 consecutive elements (inside one tensor, and inside one row of a
// row-sparse tensor), a warp per block, and chunks of 8 blocks are handed out
// to a grid of resident thread blocks in turn.  The list's descriptors are
// kernel parameters, so a step needs no copy to the device and can be
// captured.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "ptx.cuh"

namespace hstu {
namespace {

constexpr int kBlockElems = HSTU_STATE_BLOCK;
constexpr int kChunkBlocks = 8;  // one per warp
constexpr int kThreads = 32 * kChunkBlocks;
// Tensors of one launch: 120 bytes each in 32,764 bytes of kernel parameters.
constexpr int kMaxTensors = 256;

// ---------------------------------------------------------------- gradient norm
struct NormTensor {
  const void* grad;
  const int64_t* n_rows;  // row-sparse: rows used (device); else null
  int64_t n;              // elements (row-sparse: of max_rows rows)
  int64_t row_len, max_rows;
  int64_t chunk0;         // first chunk of this tensor
  int32_t dtype;
};
constexpr int kNormChunk = 4096;
constexpr int kNormThreads = 256;

struct NormArgs {
  NormTensor t[kMaxTensors];
  int n;
  int64_t chunks;
  double* part;  // [gridDim.x]
  int* status;
};

struct NormFinal {
  const double* part;
  int parts;
  double max_norm;
  float* out;
};

DEVI void add_squares(double& acc, int dtype, const uint4& r) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dtype == HSTU_FP32) {
      const double x = __uint_as_float(w[i]);
      acc = fma(x, x, acc);
    } else {
      float2 f;
      if (dtype == HSTU_BF16) {
        f.x = __uint_as_float(w[i] << 16);
        f.y = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      }
      const double x = f.x, y = f.y;
      acc = fma(x, x, acc);
      acc = fma(y, y, acc);
    }
  }
}
DEVI float load_elem(int dtype, const void* p, int64_t i) {
  return dtype == HSTU_FP32   ? static_cast<const float*>(p)[i]
         : dtype == HSTU_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                              : __half2float(static_cast<const __half*>(p)[i]);
}

DEVI double block_sum(double x, double* s_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_down_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = x;
  __syncthreads();
  double sum = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += s_warp[w];
  return sum;
}

// Sum of squares, one partial sum per thread block.  Squares and sums are
// fp64: a gradient of any finite fp32 size neither overflows nor vanishes,
// and at 4 bytes a gradient the fp64 units keep up with the memory.
__global__ void __launch_bounds__(kNormThreads)
    k_norm_part(const __grid_constant__ NormArgs a) {
  __shared__ double s_warp[kNormThreads / 32];
  grid_dep_launch();
  double acc = 0;
  int t = 0;
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    while (t + 1 < a.n && c >= a.t[t + 1].chunk0) ++t;
    const NormTensor& q = a.t[t];
    int64_t n = q.n;
    if (q.n_rows) {
      n = min(max(*q.n_rows, (int64_t)0), q.max_rows) * q.row_len;
    }
    const int64_t e0 = (c - q.chunk0) * kNormChunk;
    const int m = (int)min((int64_t)kNormChunk, n - e0);  // may be <= 0
    const int per = q.dtype == HSTU_FP32 ? 4 : 8;
    const int vecs = m > 0 ? m / per : 0;
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const uint8_t*>(q.grad) + e0 * (q.dtype == HSTU_FP32 ? 4 : 2));
    uint4 r[kNormChunk / 4 / kNormThreads];
#pragma unroll
    for (int u = 0; u < kNormChunk / 4 / kNormThreads; ++u) {
      const int v = u * kNormThreads + threadIdx.x;
      r[u] = v < vecs ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kNormChunk / 4 / kNormThreads; ++u) add_squares(acc, q.dtype, r[u]);
    const int tail = vecs * per + threadIdx.x;
    if (threadIdx.x < 8 && tail < m) {
      const double x = load_elem(q.dtype, q.grad, e0 + tail);
      acc = fma(x, x, acc);
    }
  }
  const double sum = block_sum(acc, s_warp);
  if (threadIdx.x == 0) a.part[blockIdx.x] = sum;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = HSTU_OK;
}

__global__ void __launch_bounds__(1024) k_norm_final(const NormFinal a) {
  __shared__ double s_warp[32];
  grid_dep_wait();
  double x = 0;
  for (int i = threadIdx.x; i < a.parts; i += blockDim.x) x += a.part[i];
  const double sum = block_sum(x, s_warp);
  if (threadIdx.x == 0) {
    const float norm = (float)sqrt(sum);
    a.out[0] = norm;
    // not finite: NaN, which makes the AdamW step leave everything as it is
    a.out[1] = !(norm <= 3.402823466e38f) ? __int_as_float(0x7fffffff)
               : norm > a.max_norm        ? (float)(a.max_norm / sqrt(sum))
                                          : 1.f;
  }
}

// ---------------------------------------------------------------- AdamW
struct StepTensor {
  const void* grad;
  void* param;
  float* master;
  __half* copy;
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  const int64_t* row_ids;  // row-sparse, else null
  const int64_t* n_rows;
  int64_t n;               // elements of the parameter
  int32_t row_len, row_blocks, max_rows;
  int32_t chunk0;          // first chunk of this tensor
  float weight_decay;
  uint8_t grad_dtype, param_dtype, state8;
};

struct StepArgs {
  StepTensor t[kMaxTensors];
  int n, first;            // tensors of this launch; number of the first one in the caller's list
  int64_t chunks;
  float b1, omb1, b2, omb2, eps;
  double log_b1, log_b2, lr;
  int64_t step;
  const int64_t* step_dev;
  const float* lr_dev;
  const float* grad_scale;
  uint64_t seed;
  int* status;
  int set_ok;              // nothing in this call can fail on the device: block 0 writes HSTU_OK
};

// The 32-bit integer mix of C. Wellons' hash prospector ("lowbias32").
DEVI uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  x *= 0x846ca68bu;
  return x ^ (x >> 16);
}
// SplitMix64's output mix (Steele, Lea and Flood, OOPSLA 2014).
DEVI uint64_t split_mix(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

// e4m3 code of the magnitude t (scaled, below 2^8 or not finite), rounded up
// when the 16-bit number r reaches the missing part: an e4m3 code step is
// 2^20 units of fp32's significand, so r * 16 is added and the rest cut.
// Below 2^-6 the codes have a fixed step, which adding 2^-6 gives them.
DEVI uint32_t e4m3_up(float t, uint32_t r16) {
  const bool sub = t < 0.015625f;
  t = sub ? __fadd_rn(t, 0.015625f) : t;
  const uint32_t c = ((__float_as_uint(t) + (r16 << 4)) >> 20) - (sub ? 968u : 960u);
  return t <= 512.f ? c : 0x7fu;  // NaN and infinity: NaN
}
DEVI float2 e4m3x2_to_f32(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
DEVI float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}
// Scale byte of a block whose largest finite magnitude is `top`: 2^(byte - 127)
// puts it into [2^7, 2^8), half of e4m3's range, so rounding up never
// saturates.
DEVI int scale_byte(float top) { return max(1, (int)(__float_as_uint(top) >> 23) - 7); }

// Four consecutive elements as fp32.
DEVI void load4(int dtype, const void* p, int64_t i, float (&f)[4]) {
  if (dtype == HSTU_FP32) {
    const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    if (dtype == HSTU_BF16) {
      f[0] = __uint_as_float(w.x << 16), f[1] = __uint_as_float(w.x & 0xffff0000u);
      f[2] = __uint_as_float(w.y << 16), f[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
      f[0] = x.x, f[1] = x.y, f[2] = y.x, f[3] = y.y;
    }
  }
}
// What storing x in `dtype` leaves of it.
DEVI float rounded(int dtype, float x) {
  return dtype == HSTU_FP32   ? x
         : dtype == HSTU_BF16 ? __bfloat162float(__float2bfloat16_rn(x))
                              : __half2float(__float2half_rn(x));
}
DEVI void store4(int dtype, void* p, int64_t i, const float (&f)[4]) {
  if (dtype == HSTU_FP32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
  } else if (dtype == HSTU_BF16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(f[0], f[1]), y = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  } else {
    const __half2 x = __floats2half2_rn(f[0], f[1]), y = __floats2half2_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
}
DEVI void store_elem(int dtype, void* p, int64_t i, float x) {
  if (dtype == HSTU_FP32)
    static_cast<float*>(p)[i] = x;
  else if (dtype == HSTU_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(x);
}

// One step of every tensor.  A warp takes a block of 256 elements; lane l
// holds elements 4 l + 128 j + (0..3), j = 0, 1, so every access of a warp is
// to consecutive addresses.  Bandwidth-bound: per element the gradient, the
// states and the (master) parameter are read once and the results written
// once; all of a lane's loads are issued before the first one is used.
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ StepArgs a) {
  __shared__ float s_lr, s_step_size, s_rbc2;
  __shared__ int s_skip;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    const int64_t step = a.step_dev ? *a.step_dev : a.step;
    const float gs = a.grad_scale ? *a.grad_scale : 1.f;
    const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
    // 1 - b^t without cancellation
    s_step_size = (float)(lr / -expm1((double)step * a.log_b1));
    s_rbc2 = (float)(1.0 / sqrt(-expm1((double)step * a.log_b2)));
    s_lr = (float)lr;
    s_skip = !(fabsf(gs) <= 3.402823466e38f) || step < 1;
    if (blockIdx.x == 0) {
      if (a.set_ok) *a.status = HSTU_OK;
      if (step < 1) atomicCAS(a.status, HSTU_OK, HSTU_ERR_INVALID_ARG);
    }
  }
  __syncthreads();
  if (s_skip) return;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const float lr = s_lr, step_size = s_step_size, rbc2 = s_rbc2;
  const int64_t step = a.step_dev ? *a.step_dev : a.step;
  int t = 0;
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    while (t + 1 < a.n && c >= a.t[t + 1].chunk0) ++t;
    const StepTensor& q = a.t[t];
    const int64_t b = (c - q.chunk0) * kChunkBlocks + warp;
    int64_t g0, p0, block;  // first gradient and parameter element, block number in the tensor
    int len;
    if (q.row_ids) {
      const int64_t i = b / q.row_blocks;
      const int j = (int)(b - i * q.row_blocks);
      const int64_t want = *q.n_rows;
      const int64_t rows = min(max(want, (int64_t)0), (int64_t)q.max_rows);
      if (b == 0 && lane == 0 && want != rows) atomicCAS(a.status, HSTU_OK, HSTU_ERR_BAD_IDS);
      if (i >= rows) continue;
      const int64_t row = q.row_ids[i];
      const bool bad = row < 0 || row >= q.n / q.row_len || (i > 0 && q.row_ids[i - 1] >= row);
      if (bad) {
        if (lane == 0) atomicCAS(a.status, HSTU_OK, HSTU_ERR_BAD_IDS);
        continue;
      }
      g0 = i * q.row_len + j * kBlockElems;
      p0 = row * q.row_len + j * kBlockElems;
      block = row * q.row_blocks + j;
      len = min(kBlockElems, q.row_len - j * kBlockElems);
    } else {
      g0 = p0 = b * kBlockElems;
      if (g0 >= q.n) continue;
      block = b;
      len = (int)min((int64_t)kBlockElems, q.n - g0);
    }
    const bool whole = len == kBlockElems && !(q.row_ids && (q.row_len & 3));
    const void* wide = q.master ? static_cast<const void*>(q.master) : q.param;
    const int wide_dt = q.master ? HSTU_FP32 : q.param_dtype;
    float g[2][4], p[2][4], m[2][4], v[2][4];
    float ms = 0.f, vs = 0.f;
    if (q.state8) {
      ms = __uint_as_float((uint32_t)q.m_scale[block] << 23);
      vs = __uint_as_float((uint32_t)q.v_scale[block] << 23);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = 4 * lane + 128 * j;
      if (whole) {
        load4(q.grad_dtype, q.grad, g0 + e, g[j]);
        load4(wide_dt, wide, p0 + e, p[j]);
        if (q.state8) {
          const uint32_t mc = *reinterpret_cast<const uint32_t*>(static_cast<uint8_t*>(q.m) + p0 + e);
          const uint32_t vc = *reinterpret_cast<const uint32_t*>(static_cast<uint8_t*>(q.v) + p0 + e);
          const float2 m0 = e4m3x2_to_f32(mc & 0xffffu), m1 = e4m3x2_to_f32(mc >> 16);
          const float2 v0 = e4m3x2_to_f32(vc & 0xffffu), v1 = e4m3x2_to_f32(vc >> 16);
          m[j][0] = m0.x, m[j][1] = m0.y, m[j][2] = m1.x, m[j][3] = m1.y;
          v[j][0] = v0.x, v[j][1] = v0.y, v[j][2] = v1.x, v[j][3] = v1.y;
        } else {
          load4(HSTU_FP32, q.m, p0 + e, m[j]);
          load4(HSTU_FP32, q.v, p0 + e, v[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = e + i < len;
          g[j][i] = in ? load_elem(q.grad_dtype, q.grad, g0 + e + i) : 0.f;
          p[j][i] = in ? load_elem(wide_dt, wide, p0 + e + i) : 0.f;
          if (q.state8) {
            const uint32_t mc = in ? static_cast<uint8_t*>(q.m)[p0 + e + i] : 0;
            const uint32_t vc = in ? static_cast<uint8_t*>(q.v)[p0 + e + i] : 0;
            m[j][i] = e4m3x2_to_f32(mc).x;
            v[j][i] = e4m3x2_to_f32(vc).x;
          } else {
            m[j][i] = in ? static_cast<float*>(q.m)[p0 + e + i] : 0.f;
            v[j][i] = in ? static_cast<float*>(q.v)[p0 + e + i] : 0.f;
          }
        }
      }
    }
    // The moments' products and sums are kept apart (no contraction), so that an 8-bit state
    // does not depend on how the compiler fuses them.
    const float decay = 1.f - lr * q.weight_decay;
    float root[2][4], top_m = 0.f, top_r = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (q.state8) {
          m[j][i] = __fmul_rn(m[j][i], ms);
          const float r = __fmul_rn(v[j][i], vs);
          v[j][i] = __fmul_rn(r, r);
        }
        const float gg = __fmul_rn(g[j][i], gs);
        m[j][i] = __fadd_rn(__fmul_rn(m[j][i], a.b1), __fmul_rn(gg, a.omb1));
        v[j][i] = __fadd_rn(__fmul_rn(v[j][i], a.b2), __fmul_rn(__fmul_rn(gg, gg), a.omb2));
        root[j][i] = __fsqrt_rn(v[j][i]);
        const float u = __fdividef(m[j][i], root[j][i] * rbc2 + a.eps);
        p[j][i] = p[j][i] * decay - u * step_size;
        top_m = fmaxf(top_m, finite_abs(m[j][i]));
        top_r = fmaxf(top_r, finite_abs(root[j][i]));
      }
    }
    uint32_t mc[2] = {0, 0}, vc[2] = {0, 0};
    if (q.state8) {
      top_m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top_m)));
      top_r = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top_r)));
      const int mb = scale_byte(top_m), vb = scale_byte(top_r);
      const float mi = __uint_as_float((uint32_t)(254 - mb) << 23);
      const float vi = __uint_as_float((uint32_t)(254 - vb) << 23);
      const uint64_t key = split_mix(
          a.seed + ((((uint64_t)step << 20) + (uint64_t)(a.first + t)) + 1) * 0x9E3779B97F4A7C15ull);
      const uint32_t base = mix32(mix32((uint32_t)block ^ (uint32_t)key) ^
                                  (uint32_t)((uint64_t)block >> 32) ^ (uint32_t)(key >> 32));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t r = mix32(base + (uint32_t)(4 * lane + 128 * j + i) * 0x9E3779B9u);
          const uint32_t cm = e4m3_up(fabsf(m[j][i]) * mi, r & 0xffffu) |
                              ((__float_as_uint(m[j][i]) >> 31) << 7);
          const uint32_t cv = e4m3_up(root[j][i] * vi, r >> 16);
          mc[j] |= cm << (8 * i);
          vc[j] |= cv << (8 * i);
        }
      }
      if (lane == 0) {
        q.m_scale[block] = (uint8_t)mb;
        q.v_scale[block] = (uint8_t)vb;
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = 4 * lane + 128 * j;
      if (whole) {
        if (q.state8) {
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(q.m) + p0 + e) = mc[j];
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(q.v) + p0 + e) = vc[j];
        } else {
          store4(HSTU_FP32, q.m, p0 + e, m[j]);
          store4(HSTU_FP32, q.v, p0 + e, v[j]);
        }
        if (q.master) store4(HSTU_FP32, q.master, p0 + e, p[j]);
        store4(q.param_dtype, q.param, p0 + e, p[j]);
        if (q.copy) {
          float f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[i] = fminf(fmaxf(rounded(q.param_dtype, p[j][i]), -65504.f), 65504.f);
          store4(HSTU_FP16, q.copy, p0 + e, f);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (e + i >= len) continue;
          const int64_t at = p0 + e + i;
          if (q.state8) {
            static_cast<uint8_t*>(q.m)[at] = (uint8_t)(mc[j] >> (8 * i));
            static_cast<uint8_t*>(q.v)[at] = (uint8_t)(vc[j] >> (8 * i));
          } else {
            static_cast<float*>(q.m)[at] = m[j][i];
            static_cast<float*>(q.v)[at] = v[j][i];
          }
          if (q.master) q.master[at] = p[j][i];
          store_elem(q.param_dtype, q.param, at, p[j][i]);
          if (q.copy)
            q.copy[at] = __float2half_rn(
                fminf(fmaxf(rounded(q.param_dtype, p[j][i]), -65504.f), 65504.f));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- host
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool dtype_ok(int32_t t) { return t == HSTU_BF16 || t == HSTU_FP32 || t == HSTU_FP16; }

hstu_status cuda_status(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return HSTU_OK;
  note_cuda_error(e, where);
  return HSTU_ERR_CUDA;
}

constexpr int64_t kMaxElems = (int64_t)1 << 40;

// The gradient's part of a descriptor; *sparse: only some rows have one.
bool grad_ok(const hstu_adamw_tensor& t, bool* sparse) {
  *sparse = t.n_rows != nullptr;
  if (t.n < 0 || t.n > kMaxElems || !dtype_ok(t.grad_dtype) || !al16(t.grad)) return false;
  if (!*sparse) return t.n == 0 || t.grad;
  if (t.row_len < 1 || t.row_len > (1 << 20) || t.max_rows < 0 || t.max_rows > 0x7fffffffll)
    return false;
  return (t.max_rows == 0 || t.grad) && (reinterpret_cast<uintptr_t>(t.n_rows) & 7) == 0;
}

int64_t up_blocks(int64_t n) { return (n + kBlockElems - 1) / kBlockElems; }
// Blocks of 256 elements that a step walks.
int64_t tensor_blocks(const hstu_adamw_tensor& t) {
  return t.row_ids ? t.max_rows * up_blocks(t.row_len) : up_blocks(t.n);
}

constexpr int kNormBlocksPerSm = 8;
constexpr int kNormMaxParts = 148 * kNormBlocksPerSm * 8;

}  // namespace
}  // namespace hstu

// ---------------------------------------------------------------- C ABI
extern "C" {

size_t hstu_grad_norm_workspace_size(void) { return 256 + (size_t)hstu::kNormMaxParts * 8; }

hstu_status hstu_grad_norm(const hstu_adamw_tensor* tensors, int32_t n_tensors, double max_norm,
                           float* out, void* ws, size_t ws_bytes, void* stream) {
  using namespace hstu;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n_tensors < 0 || (n_tensors > 0 && !tensors) || !out || !al16(out) || !(max_norm > 0))
    return HSTU_ERR_INVALID_ARG;
  if (n_tensors > HSTU_MAX_TENSORS) return HSTU_ERR_UNSUPPORTED;
  bool sparse;
  for (int i = 0; i < n_tensors; ++i)
    if (!grad_ok(tensors[i], &sparse)) return HSTU_ERR_INVALID_ARG;
  if (!ws || ws_bytes < hstu_grad_norm_workspace_size() || !al256(ws)) return HSTU_ERR_WORKSPACE;
  double* part = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + 256);
  const int launches = std::max(1, (n_tensors + kMaxTensors - 1) / kMaxTensors);
  const int most = std::min(num_sms() * kNormBlocksPerSm, kNormMaxParts / launches);
  int parts = 0;
  for (int l = 0; l < launches; ++l) {
    NormArgs a;
    a.n = 0;
    a.chunks = 0;
    for (int i = l * kMaxTensors; i < std::min(n_tensors, (l + 1) * kMaxTensors); ++i) {
      const hstu_adamw_tensor& t = tensors[i];
      grad_ok(t, &sparse);
      NormTensor& q = a.t[a.n];
      q.n = sparse ? t.max_rows * t.row_len : t.n;
      if (q.n == 0) continue;
      q.grad = t.grad;
      q.n_rows = t.n_rows;
      q.row_len = t.row_len;
      q.max_rows = t.max_rows;
      q.dtype = t.grad_dtype;
      q.chunk0 = a.chunks;
      a.chunks += (q.n + kNormChunk - 1) / kNormChunk;
      ++a.n;
    }
    a.part = part + parts;
    a.status = static_cast<int*>(ws);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(a.chunks, most));
    parts += grid;
    LaunchScope ls(K_GRAD_NORM, s);
    k_norm_part<<<grid, kNormThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_status(e, "hstu_grad_norm");
  }
  NormFinal f{part, parts, max_norm, out};
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  LaunchScope ls(K_GRAD_NORM, s);
  return cuda_status(cudaLaunchKernelEx(&cfg, k_norm_final, f), "hstu_grad_norm");
}

size_t hstu_adamw_workspace_size(void) { return 256; }

hstu_status hstu_adamw_step(const hstu_adamw_args* args, const hstu_adamw_tensor* tensors,
                            int32_t n_tensors, void* ws, size_t ws_bytes, void* stream) {
  using namespace hstu;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!args || n_tensors < 0 || (n_tensors > 0 && !tensors)) return HSTU_ERR_INVALID_ARG;
  if (n_tensors > HSTU_MAX_TENSORS) return HSTU_ERR_UNSUPPORTED;
  const hstu_adamw_args& h = *args;
  if (!(h.beta1 >= 0 && h.beta1 < 1) || !(h.beta2 >= 0 && h.beta2 < 1) || !(h.eps > 0) ||
      !std::isfinite(h.eps) || !std::isfinite(h.lr) || (!h.step_dev && h.step < 1))
    return HSTU_ERR_INVALID_ARG;
  bool fails = h.step_dev != nullptr;
  int64_t blocks = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const hstu_adamw_tensor& t = tensors[i];
    bool sparse;
    if (!grad_ok(t, &sparse)) return HSTU_ERR_INVALID_ARG;
    if (sparse != (t.row_ids != nullptr) || !dtype_ok(t.param_dtype) ||
        !std::isfinite(t.weight_decay) || (t.state_bits != 32 && t.state_bits != 8))
      return HSTU_ERR_INVALID_ARG;
    if (sparse && t.n % t.row_len != 0) return HSTU_ERR_INVALID_ARG;
    if (!al16(t.param) || !al16(t.master) || !al16(t.copy_f16) || !al16(t.m) || !al16(t.v) ||
        !al16(t.row_ids))
      return HSTU_ERR_INVALID_ARG;
    if (t.n > 0 && (!t.param || !t.m || !t.v)) return HSTU_ERR_INVALID_ARG;
    if (t.n > 0 && t.state_bits == 8 && (!t.m_scale || !t.v_scale)) return HSTU_ERR_INVALID_ARG;
    fails |= sparse;
    blocks += tensor_blocks(t) + kChunkBlocks;
  }
  if (blocks / kChunkBlocks > 0x7fffffffll) return HSTU_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < hstu_adamw_workspace_size() || !al256(ws)) return HSTU_ERR_WORKSPACE;
  if (fails) {
    const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int), s);
    if (e != cudaSuccess) return cuda_status(e, "hstu_adamw_step");
  }
  StepArgs a;
  a.b1 = (float)h.beta1;
  a.omb1 = (float)(1.0 - h.beta1);
  a.b2 = (float)h.beta2;
  a.omb2 = (float)(1.0 - h.beta2);
  a.eps = (float)h.eps;
  a.log_b1 = std::log(h.beta1);
  a.log_b2 = std::log(h.beta2);
  a.lr = h.lr;
  a.step = h.step;
  a.step_dev = h.step_dev;
  a.lr_dev = h.lr_dev;
  a.grad_scale = h.grad_scale;
  a.seed = h.seed;
  a.status = static_cast<int*>(ws);
  a.set_ok = !fails;
  int i = 0;
  do {
    a.first = i;
    a.n = 0;
    a.chunks = 0;
    for (; i < n_tensors && a.n < kMaxTensors; ++i) {
      const hstu_adamw_tensor& t = tensors[i];
      StepTensor& q = a.t[a.n++];
      q.grad = t.grad;
      q.param = t.param;
      q.master = t.param_dtype == HSTU_FP32 ? nullptr : t.master;
      q.copy = static_cast<__half*>(t.copy_f16);
      q.m = t.m;
      q.v = t.v;
      q.m_scale = t.m_scale;
      q.v_scale = t.v_scale;
      q.row_ids = t.row_ids;
      q.n_rows = t.n_rows;
      q.n = t.n;
      q.row_len = t.row_ids ? (int32_t)t.row_len : 0;
      q.row_blocks = t.row_ids ? (int32_t)up_blocks(t.row_len) : 0;
      q.max_rows = (int32_t)t.max_rows;
      q.chunk0 = (int32_t)a.chunks;
      q.weight_decay = (float)t.weight_decay;
      q.grad_dtype = (uint8_t)t.grad_dtype;
      q.param_dtype = (uint8_t)t.param_dtype;
      q.state8 = t.state_bits == 8;
      a.chunks += (tensor_blocks(t) + kChunkBlocks - 1) / kChunkBlocks;
    }
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(a.chunks, num_sms() * 8));
    LaunchScope ls(K_ADAMW, s);
    k_adamw<<<grid, kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_status(e, "hstu_adamw_step");
  } while (i < n_tensors);
  return HSTU_OK;
}

}  // extern "C"
