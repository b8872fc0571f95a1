// optim.cu — the global gradient norm and the AdamW step over many tensors.
//
// Both walk a list of tensors in one launch: the list is cut into blocks of
// 256 consecutive elements (inside one tensor, and inside one row of a
// row-sparse tensor), a warp per block, and chunks of blocks are handed out to
// a grid of resident thread blocks in turn.  The list's descriptors are
// kernel parameters, so a step needs no copy to the device and can be
// captured.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "ptx.cuh"

namespace hstu {
namespace {

constexpr int kBlockElems = HSTU_STATE_BLOCK;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Tensors of one launch: 120 bytes each, in 32,764 bytes of kernel parameters.
// A short list takes kernels with fewer parameters: copying 30 KB of them costs
// the launching thread about 2 us.
constexpr int kMaxTensors = 256, kFewTensors = 32;

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

template <int N>
struct NormArgs {
  NormTensor t[N];
  int n;
  int64_t chunks;
  double* part;  // [gridDim.x]
  int* status;
  double max_norm;  // one-launch form only, with out and after
  float* out;
  const int* after;
};

struct NormFinal {
  const double* part;
  int parts;
  double max_norm;
  float* out;
  const int* after;  // status word of the call that made the gradients, or null
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

// Sum over the block, in every thread; x summed in a fixed order.
DEVI double block_sum(double x, double* s_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_down_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = x;
  __syncthreads();
  double sum = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += s_warp[w];
  return sum;
}

DEVI void write_norm(double sum, double max_norm, float* out, const int* after) {
  // a failed call left its gradients unwritten, or partly written: whatever they add up to, no norm
  const float norm = after && *after != HSTU_OK ? __int_as_float(0x7fffffff) : (float)sqrt(sum);
  out[0] = norm;
  // not finite: NaN, which makes the AdamW step leave everything as it is
  out[1] = !(norm <= 3.402823466e38f) ? __int_as_float(0x7fffffff)
           : norm > max_norm          ? (float)(max_norm / sqrt(sum))
                                      : 1.f;
}

// Sum of squares of the chunks that fall to this group of kNormThreads
// threads, one of `groups`; U chunks are read before the first one is used.
// Squares and sums are fp64: a gradient of any finite fp32 size neither
// overflows nor vanishes, and at 4 bytes a gradient the fp64 units keep up with
// the memory (four sums per thread, so that one addition need not wait for the
// one before).
template <int U, int N>
DEVI double sum_chunks(const NormArgs<N>& a, int64_t group, int64_t groups) {
  constexpr int kVecs = kNormChunk / 4 / kNormThreads;
  const int tid = threadIdx.x % kNormThreads;
  double acc[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u) acc[u] = 0;
  int t = 0;
  for (int64_t c0 = group; c0 < a.chunks; c0 += groups * U) {
    uint4 r[U][kVecs];
    int dtype[U];
    float last[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t c = c0 + k * groups;
      const bool in = c < a.chunks;
      while (in && t + 1 < a.n && c >= a.t[t + 1].chunk0) ++t;
      const NormTensor& q = a.t[t];
      dtype[k] = q.dtype;
      int64_t n = q.n;
      if (q.n_rows) n = min(max(*q.n_rows, (int64_t)0), q.max_rows) * q.row_len;
      const int64_t e0 = (c - q.chunk0) * kNormChunk;
      // elements of this chunk that count; none behind a row-sparse gradient's rows in use, which
      // may lie more than 2^31 elements before the chunk
      const int m = in && e0 < n ? (int)min((int64_t)kNormChunk, n - e0) : 0;
      const int per = dtype[k] == HSTU_FP32 ? 4 : 8;
      const int vecs = m > 0 ? m / per : 0;  // (m is not negative, but asking saves 1.2 of 39 us)
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint8_t*>(q.grad) + e0 * (dtype[k] == HSTU_FP32 ? 4 : 2));
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int v = u * kNormThreads + tid;
        r[k][u] = v < vecs ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
      }
      const int tail = vecs * per + tid;
      last[k] = tid < 8 && tail < m ? load_elem(dtype[k], q.grad, e0 + tail) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) add_squares(acc[u], dtype[k], r[k][u]);
      const double x = last[k];
      acc[0] = fma(x, x, acc[0]);
    }
  }
  double sum = 0;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) sum += acc[u];
  return sum;
}

// One partial sum per thread block.
template <int N>
__global__ void __launch_bounds__(kNormThreads)
    k_norm_part(const __grid_constant__ NormArgs<N> a) {
  __shared__ double s_warp[kNormThreads / 32];
  grid_dep_launch();
  const double sum = block_sum(sum_chunks<2>(a, blockIdx.x, gridDim.x), s_warp);
  if (threadIdx.x == 0) a.part[blockIdx.x] = sum;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = HSTU_OK;
}

__global__ void __launch_bounds__(1024) k_norm_final(const NormFinal a) {
  __shared__ double s_warp[32];
  grid_dep_wait();
  double x = 0;
  for (int i = threadIdx.x; i < a.parts; i += blockDim.x) x += a.part[i];
  const double sum = block_sum(x, s_warp);
  if (threadIdx.x == 0) write_norm(sum, a.max_norm, a.out, a.after);
}

// The whole norm in one launch, by one cluster of 16 blocks, where that is
// little work: a second launch costs the host more than the other SMs would
// save (up to 4 MB of gradients).
constexpr int kNormCluster = 16;
constexpr int kNormGroups = 4;  // groups of kNormThreads threads per block
template <int N>
__global__ void __launch_bounds__(kNormThreads * kNormGroups)
    k_norm_small(const __grid_constant__ NormArgs<N> a) {
  namespace cg = cooperative_groups;
  __shared__ double s_warp[kNormThreads * kNormGroups / 32], s_sum;
  cg::cluster_group cluster = cg::this_cluster();
  const int block = (int)cluster.block_rank();
  const double x = sum_chunks<2>(a, block * kNormGroups + threadIdx.x / kNormThreads,
                                 kNormCluster * kNormGroups);
  const double sum = block_sum(x, s_warp);
  if (threadIdx.x == 0) s_sum = sum;
  cluster.sync();
  if (block == 0 && threadIdx.x < 32) {
    const double x =
        threadIdx.x < kNormCluster ? *cluster.map_shared_rank(&s_sum, threadIdx.x) : 0;
    double all = 0;
#pragma unroll
    for (int r = 0; r < kNormCluster; ++r) all += __shfl_sync(0xffffffffu, x, r);
    if (threadIdx.x == 0) {
      write_norm(all, a.max_norm, a.out, a.after);
      *a.status = HSTU_OK;
    }
  }
  cluster.sync();  // no block leaves while its sum is read
}

// ---------------------------------------------------------------- AdamW
struct StepTensor {
  const void* grad;
  void* param;
  void* master;
  __half* copy;
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  const int64_t* row_ids;  // row-sparse, else null
  const int64_t* n_rows;
  int64_t n;               // elements of the parameter
  int64_t rows;            // row-sparse: rows of the table
  int32_t row_len, row_blocks, max_rows;
  int32_t chunk0;          // first chunk of this tensor
  float weight_decay;
  uint8_t grad_dtype, param_dtype;
  uint8_t per;             // consecutive blocks that a warp takes (<= 16)
  uint8_t kind;            // kTypes * (8-bit states) + its Types
};

template <int N>
struct StepArgs {
  StepTensor t[N];
  int n, first;            // tensors of this launch; number of the first one in the caller's list
  int64_t chunks;
  float b1, omb1, b2, omb2, eps;
  double log_b1, log_b2, bc1, bc2, lr;
  int64_t step;
  const int64_t* step_dev;
  const float* lr_dev;
  const float* grad_scale;
  uint64_t seed;
  int* status;
  int set_ok;              // nothing in this call can fail on the device: block 0 writes HSTU_OK
};

static_assert(sizeof(StepArgs<kMaxTensors>) <= 32764, "kernel parameters");

// The 32-bit integer mix of C. Wellons' hash prospector ("lowbias32").
DEVI uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  x *= 0x846ca68bu;
  return x ^ (x >> 16);
}
constexpr uint64_t kGolden = 0x9E3779B97F4A7C15ull;
// SplitMix64's output mix (Steele, Lea and Flood, OOPSLA 2014).
DEVI uint64_t split_mix(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

// e4m3 code of the magnitude of x = 2^-120 t, |t| < 2^8, rounded up when the
// 16-bit number r / 2^16 reaches the missing part.  The factor turns fp32's
// exponent field into e4m3's (bias 127 - 120 = 7) and its subnormal numbers
// into e4m3's (both have the fixed step of the smallest exponent), so the code
// is what lies above the lowest 20 bits, and r * 16 is added before they are
// cut.  Everything is 4 bits further up, so that the sign falls off and the
// code is the top byte; r8 is r shifted left by 8.
constexpr float kCodeScale = 7.5231638452626400e-37f;  // 2^-120
DEVI uint32_t e4m3_up(float x, uint32_t r8) { return (__float_as_uint(x) << 4) + r8; }
// Top bytes of four words.
DEVI uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}
DEVI float2 e4m3x2_to_f32(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
constexpr uint32_t kInfBits = 0x7f800000u;
DEVI uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// The larger magnitude of the two, NaN if one is (its sign means nothing).
DEVI float max_abs(float a, float b) {
  float y;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// 1 / x to one ulp, x normal.
DEVI float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Scale byte of a block whose largest finite magnitude has these bits:
// 2^(byte - 127) puts it into [2^7, 2^8), half of e4m3's range, so rounding up
// never saturates.
DEVI int scale_byte(uint32_t top) { return max(1, (int)(top >> 23) - 7); }
DEVI float scale_inverse(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// Four consecutive elements as they lie in memory (16-bit types: x and y).
DEVI uint4 raw4(bool wide, const uint8_t* p, int e) {
  if (wide) return *reinterpret_cast<const uint4*>(p + 4 * e);
  const uint2 w = *reinterpret_cast<const uint2*>(p + 2 * e);
  return make_uint4(w.x, w.y, 0, 0);
}
DEVI uint4 wide2(const uint4* p, int i) {
  const uint2 w = reinterpret_cast<const uint2*>(p)[i];
  return make_uint4(w.x, w.y, 0, 0);
}
DEVI void widen4(int dtype, const uint4& r, float (&f)[4]) {
  if (dtype == HSTU_FP32) {
    f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
  } else if (dtype == HSTU_BF16) {
    f[0] = __uint_as_float(r.x << 16), f[1] = __uint_as_float(r.x & 0xffff0000u);
    f[2] = __uint_as_float(r.y << 16), f[3] = __uint_as_float(r.y & 0xffff0000u);
  } else {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
    f[0] = x.x, f[1] = x.y, f[2] = y.x, f[3] = y.y;
  }
}
DEVI uint32_t bits2(const __nv_bfloat162& x) { return *reinterpret_cast<const uint32_t*>(&x); }
DEVI uint32_t bits2(const __half2& x) { return *reinterpret_cast<const uint32_t*>(&x); }
// What storing x in `dtype` leaves of it.
DEVI float rounded(int dtype, float x) {
  return dtype == HSTU_FP32   ? x
         : dtype == HSTU_BF16 ? __bfloat162float(__float2bfloat16_rn(x))
                              : __half2float(__float2half_rn(x));
}
DEVI void store_elem(int dtype, void* p, int64_t i, float x) {
  if (dtype == HSTU_FP32)
    static_cast<float*>(p)[i] = x;
  else if (dtype == HSTU_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(x);
}

// Two fp32 operations in one instruction, each rounded as the single one.  The
// 8-bit step is bound by the instructions it issues: with these and a shorter
// encoding 42M parameters take 141 instead of 147 us, and 152 instead of 161
// under the power limit.
DEVI float2 both(float x) { return make_float2(x, x); }
DEVI float2 mul2(float2 x, float2 y) {
  float2 z;
  asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\n"
      "mul.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;\n}"
      : "=f"(z.x), "=f"(z.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return z;
}
DEVI float2 fma2(float2 x, float2 y, float2 w) {
  float2 z;
  asm("{\n.reg .b64 x, y, w, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\n"
      "mov.b64 w, {%6, %7};\nfma.rn.f32x2 z, x, y, w;\nmov.b64 {%0, %1}, z;\n}"
      : "=f"(z.x), "=f"(z.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(w.x), "f"(w.y));
  return z;
}

// What all elements of a step share.
struct StepConst {
  float b1, omb1, b2, omb2, eps, gs, step_size, rbc2, decay;
};

// m and v after the step.  Products and sums are kept apart (no contraction),
// so that an 8-bit state does not depend on how the compiler fuses them; the
// sums are single instructions because add.rn.f32x2 behind mul.rn.f32x2 does
// get fused (seen in the results).
DEVI float2 add_apart(float2 x, float2 y) {
  return make_float2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}
DEVI void moments(const StepConst& k, float2 g, float2& m, float2& v) {
  g = mul2(g, both(k.gs));
  m = add_apart(mul2(m, both(k.b1)), mul2(g, both(k.omb1)));
  v = add_apart(mul2(v, both(k.b2)), mul2(mul2(g, g), both(k.omb2)));
}
// The new parameters; eps >= 2^-126, so the denominator is a normal number.
DEVI float2 new_param(const StepConst& k, float2 p, float2 m, float2 root) {
  const float2 d = fma2(root, both(k.rbc2), both(k.eps));
  const float2 step =
      mul2(mul2(m, make_float2(rcp_approx(d.x), rcp_approx(d.y))), both(k.step_size));
  return fma2(fma2(p, both(k.decay), step), both(-1.f), p);
}

// Key of a block's random numbers, and an element's 32 random bits: the low
// half is m's number, the high half r's.
DEVI uint32_t block_key(uint64_t key, int64_t block) {
  return mix32(mix32((uint32_t)block ^ (uint32_t)key) ^ (uint32_t)((uint64_t)block >> 32) ^
               (uint32_t)(key >> 32));
}
DEVI uint32_t elem_random(uint32_t base, int e) { return mix32(base + (uint32_t)e * 0x9E3779B9u); }
DEVI uint32_t low16_up(uint32_t r) { return __byte_perm(r, 0, 0x4104); }   // << 8
DEVI uint32_t high16_up(uint32_t r) { return __byte_perm(r, 0, 0x4324); }

// Where a block of up to 256 elements lies.
struct BlockAt {
  int64_t g0, p0, block;  // first gradient and parameter element, block number in the tensor
  int len;
};

// Types of a tensor that the loop need not ask for: kWide, the gradient and the
// parameter that is read (the master, or the parameter itself) are fp32, as
// this library's backward pass and trainer have them; kTable, fp32 gradients of
// a bf16 parameter without a master (an embedding table).  With the questions
// in the loop its code no longer fits the instruction cache next to the SM's
// partitions: touched rows of 8-bit states 27 us instead of 31.
enum Types { kAny = 0, kWide = 1, kTable = 2, kTypes = 3 };
template <int TY>
DEVI bool grad_wide(const StepTensor& q) { return TY != kAny || q.grad_dtype == HSTU_FP32; }
template <int TY>
DEVI bool param_wide(const StepTensor& q) {
  return TY == kWide || (TY == kAny && (q.master || q.param_dtype == HSTU_FP32));
}
template <int TY>
DEVI int param_type(const StepTensor& q) { return TY == kTable ? HSTU_BF16 : q.param_dtype; }

// Stores four new parameters and what is kept of them.
template <int TY>
DEVI void store_param(const StepTensor& q, int64_t at, const float (&p)[4]) {
  if (param_wide<TY>(q))
    *reinterpret_cast<float4*>(static_cast<float*>(q.master ? q.master : q.param) + at) =
        make_float4(p[0], p[1], p[2], p[3]);
  float2 x = make_float2(p[0], p[1]), y = make_float2(p[2], p[3]);  // as stored
  if (param_type<TY>(q) == HSTU_BF16) {
    const __nv_bfloat162 s = __floats2bfloat162_rn(x.x, x.y), t = __floats2bfloat162_rn(y.x, y.y);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(q.param) + at) =
        make_uint2(bits2(s), bits2(t));
    x = __bfloat1622float2(s), y = __bfloat1622float2(t);
  } else if (param_type<TY>(q) == HSTU_FP16) {
    const __half2 s = __floats2half2_rn(x.x, x.y), t = __floats2half2_rn(y.x, y.y);
    *reinterpret_cast<uint2*>(static_cast<__half*>(q.param) + at) = make_uint2(bits2(s), bits2(t));
    x = __half22float2(s), y = __half22float2(t);
  }
  if (q.copy) *reinterpret_cast<uint2*>(q.copy + at) = make_uint2(pack_f16x2_sat(x.x, x.y), pack_f16x2_sat(y.x, y.y));
}

// 8-bit states: a whole block of 256 elements as it lies in memory, copied into
// shared memory one block ahead of the arithmetic (two stages per warp).  The
// arithmetic is long enough that a warp's loads have to be in flight
// meanwhile, and has no registers to hold them: 160 -> 146 us for 42M
// parameters when it was added.  (fp32 states: 224 us against 218 without it.)
struct Stage {
  uint4 g[64], p[64], m[16], v[16];  // 16-bit gradients and parameters: half
};

template <int TY>
DEVI void stage_block(const StepTensor& q, const BlockAt& at, Stage& s) {
  const int lane = threadIdx.x & 31;
  const bool gw = grad_wide<TY>(q), pw = param_wide<TY>(q);
  const uint8_t* gp = static_cast<const uint8_t*>(q.grad) + (at.g0 << (gw ? 2 : 1)) + 16 * lane;
  const uint8_t* wp = static_cast<const uint8_t*>(q.master ? q.master : q.param) +
                      (at.p0 << (pw ? 2 : 1)) + 16 * lane;
  const uint8_t* cp = static_cast<const uint8_t*>(lane < 16 ? q.m : q.v) + at.p0 + 16 * (lane & 15);
  copy16(&s.g[lane], gp);
  if (gw) copy16(&s.g[32 + lane], gp + 512);
  copy16(&s.p[lane], wp);
  if (pw) copy16(&s.p[32 + lane], wp + 512);
  copy16((lane < 16 ? s.m : s.v) + (lane & 15), cp);
}

// The step of one block whose length is a multiple of 4 and whose rows are
// 16-byte aligned.  WHOLE: 256 elements; with 8-bit states staged.  Lane l
// holds elements 4 l + 128 j + (0..3), j = 0, 1, so every access of a warp is to
// consecutive addresses; all of a lane's loads are issued before the first one
// is used.  8-bit states: the block's scale bytes are `bytes` of lanes u (m) and
// 16 + u (v), and are replaced by the new ones.
template <bool S8, int TY, bool WHOLE>
DEVI void step_block(const StepTensor& q, const BlockAt& at, const StepConst& k, uint64_t key,
                     int u, int& bytes, const Stage* st) {
  const int lane = threadIdx.x & 31;
  const bool gw = grad_wide<TY>(q), pw = param_wide<TY>(q);
  const uint8_t* gp = static_cast<const uint8_t*>(q.grad) + (at.g0 << (gw ? 2 : 1));
  const uint8_t* wp = static_cast<const uint8_t*>(q.master ? q.master : q.param) +
                      (at.p0 << (pw ? 2 : 1));
  uint8_t* mp = static_cast<uint8_t*>(q.m) + (S8 ? at.p0 : 4 * at.p0);
  uint8_t* vp = static_cast<uint8_t*>(q.v) + (S8 ? at.p0 : 4 * at.p0);
  uint4 gr[2], pr[2], mr[2], vr[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 4 * lane + 128 * j, x = lane + 32 * j;
    if (S8 && WHOLE) {
      gr[j] = gw ? st->g[x] : wide2(st->g, x);
      pr[j] = pw ? st->p[x] : wide2(st->p, x);
      mr[j].x = reinterpret_cast<const uint32_t*>(st->m)[x];
      vr[j].x = reinterpret_cast<const uint32_t*>(st->v)[x];
      continue;
    }
    if (!WHOLE && e >= at.len) {
      gr[j] = pr[j] = mr[j] = vr[j] = make_uint4(0, 0, 0, 0);
      continue;
    }
    gr[j] = raw4(gw, gp, e);
    pr[j] = raw4(pw, wp, e);
    if (S8) {
      mr[j].x = *reinterpret_cast<const uint32_t*>(mp + e);
      vr[j].x = *reinterpret_cast<const uint32_t*>(vp + e);
    } else {
      mr[j] = raw4(true, mp, e);
      vr[j] = raw4(true, vp, e);
    }
  }
  float ms = 0.f, vs = 0.f;
  if (S8) {
    ms = __uint_as_float((uint32_t)__shfl_sync(0xffffffffu, bytes, u) << 23);
    vs = __uint_as_float((uint32_t)__shfl_sync(0xffffffffu, bytes, 16 + u) << 23);
  }
  float m[2][4], v[2][4], top_m = 0.f, top_r = 0.f;  // 8-bit states: v becomes the root
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 4 * lane + 128 * j;
    float g[4], p[4];
    widen4(TY != kAny ? HSTU_FP32 : q.grad_dtype, gr[j], g);
    widen4(pw ? HSTU_FP32 : param_type<TY>(q), pr[j], p);
    if (!S8) {
      widen4(HSTU_FP32, mr[j], m[j]);
      widen4(HSTU_FP32, vr[j], v[j]);
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      float2 m2, v2;
      if (S8) {
        m2 = mul2(e4m3x2_to_f32(mr[j].x >> (8 * i) & 0xffffu), both(ms));
        v2 = mul2(e4m3x2_to_f32(vr[j].x >> (8 * i) & 0xffffu), both(vs));
        v2 = mul2(v2, v2);
      } else {
        m2 = make_float2(m[j][i], m[j][i + 1]);
        v2 = make_float2(v[j][i], v[j][i + 1]);
      }
      moments(k, make_float2(g[i], g[i + 1]), m2, v2);
      const float2 root = make_float2(__fsqrt_rn(v2.x), __fsqrt_rn(v2.y));
      const float2 p2 = new_param(k, make_float2(p[i], p[i + 1]), m2, root);
      p[i] = p2.x, p[i + 1] = p2.y;
      m[j][i] = m2.x, m[j][i + 1] = m2.y;
      v[j][i] = S8 ? root.x : v2.x, v[j][i + 1] = S8 ? root.y : v2.y;
      if (S8) {
        top_m = max_abs(max_abs(top_m, m2.x), m2.y);
        top_r = max_abs(max_abs(top_r, root.x), root.y);
      }
    }
    if (!WHOLE && e >= at.len) continue;
    if (!S8) {
      *reinterpret_cast<float4*>(mp + 4 * e) = make_float4(m[j][0], m[j][1], m[j][2], m[j][3]);
      *reinterpret_cast<float4*>(vp + 4 * e) = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
    }
    store_param<TY>(q, at.p0 + e, p);
  }
  if (!S8) return;
  uint32_t tm = __reduce_max_sync(0xffffffffu, abs_bits(top_m));
  uint32_t tr = __reduce_max_sync(0xffffffffu, abs_bits(top_r));
  uint32_t m_nan[2] = {0, 0}, v_nan[2] = {0, 0};  // codes of what is not finite
  if (tm >= kInfBits || tr >= kInfBits) {          // the same for the whole warp; rare
    tm = tr = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (abs_bits(m[j][i]) >= kInfBits) {
          m_nan[j] |= (0x7fu | ((__float_as_uint(m[j][i]) >> 24) & 0x80u)) << (8 * i);
          m[j][i] = 0.f;
        }
        if (abs_bits(v[j][i]) >= kInfBits) {
          v_nan[j] |= 0x7fu << (8 * i);
          v[j][i] = 0.f;
        }
        tm = max(tm, abs_bits(m[j][i]));
        tr = max(tr, abs_bits(v[j][i]));
      }
    }
    tm = __reduce_max_sync(0xffffffffu, tm);
    tr = __reduce_max_sync(0xffffffffu, tr);
  }
  const int m_byte = scale_byte(tm), v_byte = scale_byte(tr);
  if ((lane & 15) == u) bytes = lane < 16 ? m_byte : v_byte;
  const float mi = scale_inverse(m_byte), vi = scale_inverse(v_byte);
  const uint32_t base = block_key(key, at.block) + (uint32_t)(4 * lane) * 0x9E3779B9u;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 4 * lane + 128 * j;
    if (!WHOLE && e >= at.len) continue;
    uint32_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      // (two factors: their product can be below fp32's range)
      const float2 x = mul2(mul2(make_float2(m[j][i], m[j][i + 1]), both(mi)), both(kCodeScale));
      const float2 y = mul2(mul2(make_float2(v[j][i], v[j][i + 1]), both(vi)), both(kCodeScale));
      const uint32_t r0 = elem_random(base, 128 * j + i), r1 = elem_random(base, 128 * j + i + 1);
      a[i] = e4m3_up(x.x, low16_up(r0)), a[i + 1] = e4m3_up(x.y, low16_up(r1));
      b[i] = e4m3_up(y.x, high16_up(r0)), b[i + 1] = e4m3_up(y.y, high16_up(r1));
    }
    const uint32_t sign = top_bytes(__float_as_uint(m[j][0]), __float_as_uint(m[j][1]),
                                    __float_as_uint(m[j][2]), __float_as_uint(m[j][3]));
    *reinterpret_cast<uint32_t*>(mp + e) =
        top_bytes(a[0], a[1], a[2], a[3]) | (sign & 0x80808080u) | m_nan[j];
    *reinterpret_cast<uint32_t*>(vp + e) = top_bytes(b[0], b[1], b[2], b[3]) | v_nan[j];
  }
}

// The same for any block (the end of a tensor, rows that are not multiples of
// 4 elements), element by element: lane l takes elements l + 32 i.
template <bool S8>
DEVI void step_block_any(const StepTensor& q, const BlockAt& at, const StepConst& k, uint64_t key) {
  const int lane = threadIdx.x & 31;
  const void* wide = q.master ? q.master : q.param;
  const int wide_dt = q.master ? HSTU_FP32 : q.param_dtype;
  float ms = 0.f, vs = 0.f, m[8], root[8];
  if (S8) {
    ms = __uint_as_float((uint32_t)q.m_scale[at.block] << 23);
    vs = __uint_as_float((uint32_t)q.v_scale[at.block] << 23);
  }
  uint32_t top_m = 0, top_r = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    m[i] = root[i] = 0.f;
    if (e >= at.len) continue;
    const int64_t x = at.p0 + e;
    float v, p = load_elem(wide_dt, wide, x);
    const float g = load_elem(q.grad_dtype, q.grad, at.g0 + e);
    if (S8) {
      m[i] = __fmul_rn(e4m3x2_to_f32(static_cast<uint8_t*>(q.m)[x]).x, ms);
      v = __fmul_rn(e4m3x2_to_f32(static_cast<uint8_t*>(q.v)[x]).x, vs);
      v = __fmul_rn(v, v);
    } else {
      m[i] = static_cast<float*>(q.m)[x];
      v = static_cast<float*>(q.v)[x];
    }
    float2 m2 = both(m[i]), v2 = both(v);
    moments(k, both(g), m2, v2);
    m[i] = m2.x, v = v2.x;
    root[i] = __fsqrt_rn(v);
    p = new_param(k, both(p), m2, both(root[i])).x;
    if (!S8) {
      static_cast<float*>(q.m)[x] = m[i];
      static_cast<float*>(q.v)[x] = v;
    }
    if (q.master) static_cast<float*>(q.master)[x] = p;
    store_elem(q.param_dtype, q.param, x, p);
    if (q.copy) {
      const float y = rounded(q.param_dtype, p);
      q.copy[x] = __ushort_as_half((unsigned short)pack_f16x2_sat(y, y));
    }
    const uint32_t a = abs_bits(m[i]), b = abs_bits(root[i]);
    top_m = max(top_m, a < kInfBits ? a : 0);
    top_r = max(top_r, b < kInfBits ? b : 0);
  }
  if (!S8) return;
  const int mb = scale_byte(__reduce_max_sync(0xffffffffu, top_m));
  const int vb = scale_byte(__reduce_max_sync(0xffffffffu, top_r));
  const float mi = scale_inverse(mb), vi = scale_inverse(vb);
  const uint32_t base = block_key(key, at.block);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    if (e >= at.len) continue;
    const uint32_t r = elem_random(base, e);
    const uint32_t a = abs_bits(m[i]) < kInfBits ? e4m3_up(m[i] * mi * kCodeScale, low16_up(r)) >> 24
                                                 : 0x7fu;
    const uint32_t b = abs_bits(root[i]) < kInfBits ? e4m3_up(root[i] * vi * kCodeScale, high16_up(r)) >> 24
                                                    : 0x7fu;
    static_cast<uint8_t*>(q.m)[at.p0 + e] =
        (uint8_t)(a | ((__float_as_uint(m[i]) >> 24) & 0x80u));
    static_cast<uint8_t*>(q.v)[at.p0 + e] = (uint8_t)b;
  }
  if (lane == 0) {
    q.m_scale[at.block] = (uint8_t)mb;
    q.v_scale[at.block] = (uint8_t)vb;
  }
}

// A warp's walk over the blocks of a row-sparse tensor: block j of row i of the
// list, the row's number asked for one block ahead.
struct RowWalk {
  int64_t i, di, rows;
  int j, dj;
  int64_t row, before;  // table row, and the one before it in the list
};
DEVI void ask_row(const StepTensor& q, RowWalk& w) {
  w.row = w.i < w.rows ? q.row_ids[w.i] : 0;
  w.before = w.i < w.rows && w.i > 0 ? q.row_ids[w.i - 1] : -1;
}
// The next block whose row is one of the table's and above the one before (the
// status is set for any other); false at the end.
DEVI bool next_block(const StepTensor& q, RowWalk& w, int* status, BlockAt& at) {
  while (w.i < w.rows) {
    const bool ok = w.row >= 0 && w.row < q.rows && w.before < w.row;
    at.g0 = w.i * q.row_len + w.j * kBlockElems;
    at.p0 = w.row * q.row_len + w.j * kBlockElems;
    at.block = w.row * q.row_blocks + w.j;
    at.len = min(kBlockElems, q.row_len - w.j * kBlockElems);
    w.i += w.di;
    w.j += w.dj;
    if (w.j >= q.row_blocks) {
      w.j -= q.row_blocks;
      ++w.i;
    }
    ask_row(q, w);
    if (ok) return true;
    if ((threadIdx.x & 31) == 0) atomicCAS(status, HSTU_OK, HSTU_ERR_BAD_IDS);
  }
  return false;
}

// One step of every tensor of the list whose states have this width and whose
// types are of this sort, a warp per block of 256 elements.  Bandwidth-bound:
// per element the gradient, the states and the (master) parameter are read
// once and the results written once.
//
// 8-bit states: a warp takes 4 consecutive blocks of a large dense tensor at a
// time and reads and writes their scale bytes together.  One block at a time,
// the bytes of a 32-byte sector were read and written by 32 warps on several
// SMs, which cost 20 to 45 us of 184 on 42M parameters.
//
// Thread blocks of 128 threads per SM, measured on 42M parameters: fp32 states
// 6 resident (80 registers, at which the form for any types, kAny, spills 40
// bytes) and 16 launched (218 us, 6.2 TB/s; 8 resident at 64
// registers 235; no more launched than resident 228: the hardware's handing
// out of thread blocks evens out what a fixed share does not).  8-bit states,
// bound by instructions as much as by memory: with fp32 gradients and
// parameters 4 resident and launched (141 us, 6.0 TB/s; 152 once the power limit
// holds the clock at 1.75 GHz; 5: 150 and 151; 8 launched 149), else, where a
// tensor is more likely a table whose rows take two dependent loads, 5 (14,011
// rows of 512: 27 us; 4 or 6: 29).
constexpr int resident(bool s8, int types) { return !s8 ? 6 : types == kWide ? 4 : 5; }

template <bool S8, int TY, int N>
__global__ void __launch_bounds__(kThreads, resident(S8, TY))
    k_adamw(const __grid_constant__ StepArgs<N> a) {
  __shared__ Stage s_stage[S8 ? kWarps : 1][2];
  __shared__ StepConst s_k;
  __shared__ float s_lr;
  __shared__ int s_skip;
  if (threadIdx.x == 0) {
    const int64_t step = a.step_dev ? *a.step_dev : a.step;
    const float gs = a.grad_scale ? *a.grad_scale : 1.f;
    const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
    // 1 - b^t without cancellation; with the step given as a number the host has done it
    const double bc1 = a.step_dev ? -expm1((double)step * a.log_b1) : a.bc1;
    const double bc2 = a.step_dev ? -expm1((double)step * a.log_b2) : a.bc2;
    s_k.b1 = a.b1, s_k.omb1 = a.omb1, s_k.b2 = a.b2, s_k.omb2 = a.omb2, s_k.eps = a.eps;
    s_k.gs = gs;
    s_k.step_size = (float)(lr / bc1);
    s_k.rbc2 = (float)(1.0 / sqrt(bc2));
    s_k.decay = 0.f;
    s_lr = (float)lr;
    s_skip = !(fabsf(gs) <= 3.402823466e38f) || step < 1;
    if (blockIdx.x == 0) {
      if (a.set_ok) *a.status = HSTU_OK;
      if (step < 1) atomicCAS(a.status, HSTU_OK, HSTU_ERR_INVALID_ARG);
    }
  }
  __syncthreads();
  if (s_skip) return;
  if (blockIdx.x == 0) {
    for (int t = threadIdx.x; t < a.n; t += kThreads) {
      if (!a.t[t].row_ids) continue;
      const int64_t want = *a.t[t].n_rows;
      if (want < 0 || want > a.t[t].max_rows) atomicCAS(a.status, HSTU_OK, HSTU_ERR_BAD_IDS);
    }
  }
  StepConst k = s_k;
  const int64_t step = a.step_dev ? *a.step_dev : a.step;
  const uint64_t key0 = a.seed + (((uint64_t)step << 20) + (uint64_t)a.first + 1) * kGolden;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t c = blockIdx.x;  // this thread block's next chunk of the list
  for (int t = 0; t < a.n; ++t) {
    const StepTensor& q = a.t[t];
    const int64_t end = t + 1 < a.n ? a.t[t + 1].chunk0 : a.chunks;
    if (c >= end) continue;
    const int per = q.per;
    int64_t b = ((c - q.chunk0) * kWarps + warp) * per;
    const int64_t next = (int64_t)gridDim.x * kWarps * per;
    c += (end - c + gridDim.x - 1) / gridDim.x * gridDim.x;
    if (q.kind != kTypes * S8 + TY) continue;
    k.decay = s_lr * q.weight_decay;
    const uint64_t key = split_mix(key0 + (uint64_t)t * kGolden);
    BlockAt at;
    // 8-bit states: lane u has the scale byte of m of block b + u, lane 16 + u that of v
    uint8_t* scale = lane < 16 ? q.m_scale : q.v_scale;
    const int su = lane & 15;
    int none = 0;
    if (!q.row_ids) {
      const int64_t whole = q.n / kBlockElems;
      at.len = kBlockElems;
      if (!S8) {
        // (one block a group, but the loop over a group is what keeps this at 218 us: as a single
        // loop it took 227)
        for (; b < whole; b += next) {
          const int n = (int)min((int64_t)per, whole - b);
          for (int u = 0; u < n; ++u) {
            at.block = b + u;
            at.g0 = at.p0 = at.block * kBlockElems;
            step_block<S8, TY, true>(q, at, k, key, 0, none, nullptr);
          }
          if (b + n == whole) break;
        }
      } else if (b < whole) {
        int n = (int)min((int64_t)per, whole - b), u = 0, stage = 0;
        int bytes = su < n ? scale[b + su] : 0;
        at.g0 = at.p0 = b * kBlockElems;
        __syncwarp();  // every lane is through with the tensor before
        stage_block<TY>(q, at, s_stage[warp][0]);
        copy_commit();
        for (bool more = true; more; stage ^= 1) {
          // the block after this one: of this group, or the first of this warp's next group
          int64_t b2 = b;
          int n2 = n, u2 = u + 1, bytes2 = bytes;
          if (u2 == n) {
            b2 = b + next;
            u2 = 0;
            more = b2 < whole;
            n2 = more ? (int)min((int64_t)per, whole - b2) : 0;
            if (su < n2) bytes2 = scale[b2 + su];
          }
          __syncwarp();  // every lane has read the stage that is filled now
          if (more) {
            at.g0 = at.p0 = (b2 + u2) * kBlockElems;
            stage_block<TY>(q, at, s_stage[warp][stage ^ 1]);
          }
          copy_commit();
          copy_wait_but_one();
          __syncwarp();
          at.block = b + u;
          at.g0 = at.p0 = at.block * kBlockElems;
          step_block<S8, TY, true>(q, at, k, key, u, bytes, &s_stage[warp][stage]);
          if (u2 == 0) {
            if (su < n) scale[b + su] = (uint8_t)bytes;
            if (b + n == whole) break;
            bytes = bytes2;
          }
          b = b2;
          n = n2;
          u = u2;
        }
      }
      // the shorter block behind the last whole one is with the warp whose turn it is
      at.len = (int)(q.n - whole * kBlockElems);
      if (at.len && whole / per == b / per) {
        at.block = whole;
        at.g0 = at.p0 = whole * kBlockElems;
        step_block_any<S8>(q, at, k, key);
      }
    } else {
      RowWalk w;
      w.rows = min(max(*q.n_rows, (int64_t)0), (int64_t)q.max_rows);
      w.di = next / q.row_blocks;
      w.dj = (int)(next - w.di * q.row_blocks);
      w.i = b / q.row_blocks;
      w.j = (int)(b - w.i * q.row_blocks);
      ask_row(q, w);
      if (S8 && q.row_len % kBlockElems == 0) {  // whole blocks, 16-byte aligned whatever the types
        bool have = next_block(q, w, a.status, at);
        int bytes = 0, bytes2 = 0, stage = 0;
        __syncwarp();
        if (have) {
          bytes = scale[at.block];
          stage_block<TY>(q, at, s_stage[warp][0]);
        }
        copy_commit();
        for (; have; stage ^= 1) {
          BlockAt at2;
          const bool more = next_block(q, w, a.status, at2);
          __syncwarp();
          if (more) {
            bytes2 = scale[at2.block];
            stage_block<TY>(q, at2, s_stage[warp][stage ^ 1]);
          }
          copy_commit();
          copy_wait_but_one();
          __syncwarp();
          step_block<S8, TY, true>(q, at, k, key, 0, bytes, &s_stage[warp][stage]);
          if (su == 0) scale[at.block] = (uint8_t)bytes;
          at = at2;
          bytes = bytes2;
          have = more;
        }
      } else {
        while (next_block(q, w, a.status, at)) {
          if (q.row_len % 4) {
            step_block_any<S8>(q, at, k, key);
            continue;
          }
          int bytes = S8 ? scale[at.block] : 0;
          if (!S8 && at.len == kBlockElems)
            step_block<S8, TY, !S8>(q, at, k, key, 0, bytes, nullptr);
          else
            step_block<S8, TY, false>(q, at, k, key, 0, bytes, nullptr);
          if (S8 && su == 0) scale[at.block] = (uint8_t)bytes;
        }
      }
    }
    if (S8) __syncwarp();  // every lane is done with the stages
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

constexpr int kPerWarp = 4;
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

constexpr int kNormBlocksPerSm = 4;
constexpr int kNormMaxParts = 148 * kNormBlocksPerSm * 8;
constexpr int64_t kNormSmallChunks = 256;  // of 4096 elements

template <int N>
hstu_status grad_norm(const hstu_adamw_tensor* tensors, int n_tensors, double max_norm,
                      const int* after, float* out, void* ws, cudaStream_t s) {
  double* part = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + 256);
  const int launches = std::max(1, (n_tensors + N - 1) / N);
  const int most = std::min(num_sms() * kNormBlocksPerSm, kNormMaxParts / launches);
  int parts = 0;
  cudaLaunchAttribute at[1];
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  for (int l = 0; l < launches; ++l) {
    NormArgs<N> a;
    a.n = 0;
    a.chunks = 0;
    for (int i = l * N; i < std::min(n_tensors, (l + 1) * N); ++i) {
      const hstu_adamw_tensor& t = tensors[i];
      NormTensor& q = a.t[a.n];
      q.n = t.n_rows ? t.max_rows * t.row_len : t.n;
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
    a.max_norm = max_norm;
    a.out = out;
    a.after = after;
    LaunchScope ls(K_GRAD_NORM, s);
    cudaError_t e;
    if (launches == 1 && a.chunks <= kNormSmallChunks) {
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = kNormCluster;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(kNormCluster);
      cfg.blockDim = dim3(kNormThreads * kNormGroups);
      if (clusters_resident(reinterpret_cast<const void*>(k_norm_small<N>), kNormCluster, cfg) > 0)
        return cuda_status(cudaLaunchKernelEx(&cfg, k_norm_small<N>, a), "hstu_grad_norm");
    }
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(a.chunks, most));
    parts += grid;
    k_norm_part<N><<<grid, kNormThreads, 0, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_status(e, "hstu_grad_norm");
  }
  NormFinal f{part, parts, max_norm, out, after};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  LaunchScope ls(K_GRAD_NORM, s);
  return cuda_status(cudaLaunchKernelEx(&cfg, k_norm_final, f), "hstu_grad_norm");
}

template <int N>
hstu_status adamw(const hstu_adamw_args& h, const hstu_adamw_tensor* tensors, int n_tensors,
                  bool fails, bool large, void* ws, cudaStream_t s) {
  StepArgs<N> a;
  a.b1 = (float)h.beta1;
  a.omb1 = (float)(1.0 - h.beta1);
  a.b2 = (float)h.beta2;
  a.omb2 = (float)(1.0 - h.beta2);
  a.eps = (float)h.eps;
  a.log_b1 = std::log(h.beta1);
  a.log_b2 = std::log(h.beta2);
  a.bc1 = -std::expm1((double)h.step * a.log_b1);
  a.bc2 = -std::expm1((double)h.step * a.log_b2);
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
    for (; i < n_tensors && a.n < N; ++i) {
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
      q.rows = t.row_ids ? t.n / t.row_len : 0;
      q.row_len = t.row_ids ? (int32_t)t.row_len : 0;
      q.row_blocks = t.row_ids ? (int32_t)up_blocks(t.row_len) : 0;
      q.max_rows = (int32_t)t.max_rows;
      q.chunk0 = (int32_t)a.chunks;
      q.weight_decay = (float)t.weight_decay;
      q.grad_dtype = (uint8_t)t.grad_dtype;
      q.param_dtype = (uint8_t)t.param_dtype;
      const int types = t.grad_dtype != HSTU_FP32                   ? kAny
                        : q.master || t.param_dtype == HSTU_FP32 ? kWide
                        : t.param_dtype == HSTU_BF16             ? kTable
                                                                 : kAny;
      q.kind = (uint8_t)(kTypes * (t.state_bits == 8) + types);
      q.per = large && t.state_bits == 8 && !t.row_ids ? kPerWarp : 1;
      const int64_t chunk = kWarps * q.per;
      a.chunks += (tensor_blocks(t) + chunk - 1) / chunk;
    }
    // a kernel per kind of tensor: one list seldom has more than one or two
    unsigned kinds = a.n == 0 ? 1u : 0u;
    for (int j = 0; j < a.n; ++j) kinds |= 1u << a.t[j].kind;
    static void (*const fn[2 * kTypes])(StepArgs<N>) = {
        k_adamw<false, kAny, N>, k_adamw<false, kWide, N>, k_adamw<false, kTable, N>,
        k_adamw<true, kAny, N>,  k_adamw<true, kWide, N>,  k_adamw<true, kTable, N>};
    for (int j = 0; j < 2 * kTypes; ++j) {
      if (!(kinds >> j & 1)) continue;
      LaunchScope ls(K_ADAMW, s);
      const int grid = (int)std::max<int64_t>(
          1, std::min<int64_t>(a.chunks, num_sms() * (j >= kTypes ? resident(true, j % kTypes) : 16)));
      fn[j]<<<grid, kThreads, 0, s>>>(a);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return cuda_status(e, "hstu_adamw_step");
    }
  } while (i < n_tensors);
  return HSTU_OK;
}

}  // namespace
}  // namespace hstu

// ---------------------------------------------------------------- C ABI
extern "C" {

size_t hstu_grad_norm_workspace_size(void) { return 256 + (size_t)hstu::kNormMaxParts * 8; }

hstu_status hstu_grad_norm_after(const hstu_adamw_tensor* tensors, int32_t n_tensors,
                                 double max_norm, const void* after, float* out, void* ws,
                                 size_t ws_bytes, void* stream) {
  using namespace hstu;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int* word = static_cast<const int*>(after);
  if (!al256(after)) return HSTU_ERR_INVALID_ARG;
  if (n_tensors < 0 || (n_tensors > 0 && !tensors) || !out || !al16(out) || !(max_norm > 0))
    return HSTU_ERR_INVALID_ARG;
  if (n_tensors > HSTU_MAX_TENSORS) return HSTU_ERR_UNSUPPORTED;
  bool sparse;
  for (int i = 0; i < n_tensors; ++i)
    if (!grad_ok(tensors[i], &sparse)) return HSTU_ERR_INVALID_ARG;
  if (!ws || ws_bytes < hstu_grad_norm_workspace_size() || !al256(ws)) return HSTU_ERR_WORKSPACE;
  return n_tensors <= kFewTensors
             ? grad_norm<kFewTensors>(tensors, n_tensors, max_norm, word, out, ws, s)
             : grad_norm<kMaxTensors>(tensors, n_tensors, max_norm, word, out, ws, s);
}

hstu_status hstu_grad_norm(const hstu_adamw_tensor* tensors, int32_t n_tensors, double max_norm,
                           float* out, void* ws, size_t ws_bytes, void* stream) {
  return hstu_grad_norm_after(tensors, n_tensors, max_norm, nullptr, out, ws, ws_bytes, stream);
}

size_t hstu_adamw_workspace_size(void) { return 256; }

hstu_status hstu_adamw_step(const hstu_adamw_args* args, const hstu_adamw_tensor* tensors,
                            int32_t n_tensors, void* ws, size_t ws_bytes, void* stream) {
  using namespace hstu;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!args || n_tensors < 0 || (n_tensors > 0 && !tensors)) return HSTU_ERR_INVALID_ARG;
  if (n_tensors > HSTU_MAX_TENSORS) return HSTU_ERR_UNSUPPORTED;
  const hstu_adamw_args& h = *args;
  if (!(h.beta1 >= 0 && h.beta1 < 1) || !(h.beta2 >= 0 && h.beta2 < 1) || !(h.eps >= 1.17549435e-38) ||
      !(h.eps <= 3.402823466e38) || !std::isfinite(h.lr) || (!h.step_dev && h.step < 1))
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
    blocks += tensor_blocks(t) + kWarps;
  }
  if (blocks / kWarps > 0x7fffffffll) return HSTU_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < hstu_adamw_workspace_size() || !al256(ws)) return HSTU_ERR_WORKSPACE;
  if (fails) {
    const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int), s);
    if (e != cudaSuccess) return cuda_status(e, "hstu_adamw_step");
  }
  // One block at a time where more would leave warps without work.  One against kPerWarp at a
  // time: 1M elements 6.4 and 7.0 us, 2M 10.0 and 9.3, 4M 15.5 and 16.7, 8M 26.5 and 27.3, 9.6M (the
  // border) 31.0 and 31.0, 42M 187 and 141.
  const bool large = blocks >= (int64_t)num_sms() * 32 * kPerWarp * 2;
  return n_tensors <= kFewTensors ? adamw<kFewTensors>(h, tensors, n_tensors, fails, large, ws, s)
                                  : adamw<kMaxTensors>(h, tensors, n_tensors, fails, large, ws, s);
}

}  // extern "C"
