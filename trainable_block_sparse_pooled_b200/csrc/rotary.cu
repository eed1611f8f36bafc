// Rotary positions (spa2_rotary in include/spa2.h): pairs of a head's row turned
// by position * frequency, forward (angle theta) and backward (angle -theta).
//
// rotary_kernel  one thread per unit of a token's row (16 bytes, or 16 bytes and their
//                partners), for all heads of the token or a run of them.
//
// Per element it reads and writes 2 bytes (bf16) and does 3 flops: bound by HBM. An angle costs
// an fp64 product and reduction and an fp32 sincospi, some 60 instructions a pair; one thread
// takes its unit through every head, so that they are paid once per token, not per head, and
// steps its pointers from head to head (recomputing 64-bit addresses made the kernel
// issue-bound: 15 instructions per element, 92 us against 68 below). One launch turns q and k,
// whose heads share their tokens' angles.
// Measured (q and k, one launch): [1, 40, 75600, 128] bf16 each 490 us = 6.3 TB/s, 0.96 of the
// measured copy rate; [1, 12, 32760, 128] each 68 us = 6.0 TB/s (4.6 waves of blocks).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace spa2 {

namespace {

struct RotaryTensor {
  const void* x;
  void* y;
  long long xs[3], ys[3];  // batch, head, token strides in elements
};

struct RotaryArgs {
  RotaryTensor t[2];
  int heads0, heads;  // heads of the first tensor, of all
  const void* pos;    // may be null: the token's index
  int pos64;
  long long ps[3];    // batch, axis, token strides in elements
  int first[SPA2_ROTARY_MAX_AXES];  // first pair of each axis (rd / 2 where there is none)
  const double* inv_freq;
  float scale, sin_sign;
  long long tokens;   // B * N
  int N, d, rd;
  // the launch: a unit is V elements turned in place, or (SPLIT) V and their V partners; the
  // units of a row are `turned` such and then copied ones
  int units, turned, step, partner;
  int per_block;  // heads of a block
  uint32_t units_mul, units_shift, n_mul, n_shift;  // x / units, x / N for x < 2^31 (shift 32: see divisor)
};

template <typename T>
SPA2_DEV T from_f32(float x);
template <>
SPA2_DEV float from_f32<float>(float x) { return x; }
template <>
SPA2_DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
SPA2_DEV __half from_f32<__half>(float x) { return __float2half_rn(x); }

// V elements moved as one access
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T e[V];
};

// cos and sin of position * inv_freq[p], both times the scale. The angle is
// counted in turns and reduced to [-1/2, 1/2] in fp64 (a far position times a
// frequency has more whole turns than fp32 has digits), then taken in fp32.
SPA2_DEV float2 cos_sin(const RotaryArgs& a, int b, int n, int p) {
  int axis = 0;
#pragma unroll
  for (int i = 1; i < SPA2_ROTARY_MAX_AXES; ++i) axis += p >= a.first[i];
  long long pos = n;
  if (a.pos) {
    const long long at = b * a.ps[0] + axis * a.ps[1] + n * a.ps[2];
    pos = a.pos64 ? static_cast<const long long*>(a.pos)[at] : static_cast<const int*>(a.pos)[at];
  }
  const double turns = static_cast<double>(pos) * (a.inv_freq[p] * 0.15915494309189533577);
  float s, c;
  sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
  return make_float2(c * a.scale, s * a.scale * a.sin_sign);
}

SPA2_DEV void turn(float x, float y, float2 cs, float& ox, float& oy) {
  ox = x * cs.x - y * cs.y;
  oy = x * cs.y + y * cs.x;
}

}  // namespace

// SPLIT: a unit is V elements and their V partners elsewhere in the row (the half layout; single
// elements of the interleaved one).
// Registers against loads in flight, measured: the interleaved units do best with four heads' loads
// together and 75 registers (three blocks an SM): 490 us at the 14B shape above; with no block count
// asked for the compiler took 66 registers and 580 us, with four blocks (64) 524, two heads at a time
// 501 to 519, eight 493 to 684. SPLIT units hold twice the angles: one head (two loads) at a time and
// four blocks an SM (64 registers) take 80 us for [1, 12, 32760, 128] twice, two heads and two blocks
// (88 registers) 109, five blocks (48, spilling) 88; units of 8 bytes do best with five.
// Loading a batch ahead of the one at work gained 3 us there and lost 20 in the interleaved form.
template <typename T, int V, bool SPLIT>
__global__ void __launch_bounds__(256, SPLIT ? (V == 8 ? 4 : 5) : 1) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int PAIRS = SPLIT ? V : V / 2;  // pairs of a unit
  constexpr int HB = SPLIT ? 1 : 4;         // heads in flight
  using VT = Vec<T, V>;
  const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
  const int token = a.units_shift < 32 ? (int)(__umulhi((uint32_t)idx, a.units_mul) >> a.units_shift)
                                       : (int)min(idx / a.units, a.tokens);
  const bool there = token < a.tokens;
  const int u = (int)(idx - (long long)token * a.units);
  const int b = a.n_shift < 32 ? (int)(__umulhi((uint32_t)token, a.n_mul) >> a.n_shift) : token, n = token - b * a.N;
  const bool copy = u >= a.turned || !there;
  const int e0 = copy ? a.rd + (u - a.turned) * V : u * a.step;
  const int e1 = e0 + a.partner;
  float2 cs[PAIRS];
  if (a.turned == a.units) {
    if (there) {
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) cs[i] = cos_sin(a, b, n, u * PAIRS + i);
    }
  } else {
    // part of the head: the warp shares the angles of its few turning threads out evenly. It counts where
    // a token has few heads (an eighth of 64 elements turned, 4 heads: 67 us a launch, 82 with every thread on
    // its own); q and k [1, 12, 32760, 128], an eighth or a quarter turned: 72 and 73 us against 73 and 75
    // interleaved, 103 and 102 against 109 and 106 in the half layout, for 61 us of bytes
    __shared__ float2 angle[8][32 * PAIRS];
    __shared__ int3 unit[8][32];
    const int w = threadIdx.x >> 5;
    const uint32_t turning = __ballot_sync(0xffffffffu, !copy);
    const int place = __popc(turning & ((1u << lane_id()) - 1u));
    if (!copy) unit[w][place] = make_int3(b, n, u * PAIRS);
    __syncwarp();
    for (int k = lane_id(); k < __popc(turning) * PAIRS; k += 32) {
      const int3 at = unit[w][k / PAIRS];
      angle[w][k] = cos_sin(a, at.x, at.y, at.z + k % PAIRS);
    }
    __syncwarp();
    if (!copy) {
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) cs[i] = angle[w][place * PAIRS + i];
    }
  }
  if (!there) return;
  const int first = blockIdx.y * a.per_block, last = min(a.heads, first + a.per_block);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {  // this block's heads of the first tensor, then of the second
    const int lo = which ? max(first - a.heads0, 0) : first;
    const int hi = which ? last - a.heads0 : min(last, a.heads0);
    const RotaryTensor& t = a.t[which];
    const T* from = static_cast<const T*>(t.x) + b * t.xs[0] + lo * t.xs[1] + n * t.xs[2];
    T* to = static_cast<T*>(t.y) + b * t.ys[0] + lo * t.ys[1] + n * t.ys[2];
#pragma unroll 1
    for (int h = lo; h < hi; h += HB) {
      VT x[HB], z[HB];
#pragma unroll
      for (int i = 0; i < HB; ++i) {
        if (h + i < hi) {
          x[i] = *reinterpret_cast<const VT*>(from + e0);
          if (SPLIT && !copy) z[i] = *reinterpret_cast<const VT*>(from + e1);
          from += t.xs[1];
        }
      }
#pragma unroll
      for (int i = 0; i < HB; ++i) {
        if (h + i < hi) {
          if (!copy) {
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) {
              T& s = x[i].e[SPLIT ? p : 2 * p];
              T& w = SPLIT ? z[i].e[p] : x[i].e[2 * p + 1];
              float ox, oy;
              turn(static_cast<float>(s), static_cast<float>(w), cs[p], ox, oy);
              s = from_f32<T>(ox);
              w = from_f32<T>(oy);
            }
            if (SPLIT) *reinterpret_cast<VT*>(to + e1) = z[i];
          }
          *reinterpret_cast<VT*>(to + e0) = x[i];
          to += t.ys[1];
        }
      }
    }
  }
}

// x / d = (x * mul >> 32) >> shift for x < 2^31: mul = ceil(2^(31 + l) / d) with 2^l the power of two
// from d on; for d = 1 it does not fit in 32 bits, and shift 32 says so
static void divisor(long long d, uint32_t& mul, uint32_t& shift) {
  uint32_t l = 0;
  while ((1LL << l) < d) ++l;
  mul = d == 1 ? 0u : (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
  shift = d == 1 ? 32u : l - 1;
}

template <typename T, int V, bool SPLIT>
static cudaError_t launch_rotary(RotaryArgs a, bool half, cudaStream_t s) {
  a.step = SPLIT && !half ? 2 : V;
  a.partner = half ? a.rd / 2 : 1;
  a.turned = a.rd / (SPLIT ? 2 * V : V);
  a.units = a.turned + (a.d - a.rd) / V;
  const long long blocks = (a.tokens * a.units + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  divisor(a.units, a.units_mul, a.units_shift);
  if (blocks * 256 > 0x7fffffffLL) a.units_shift = 32;
  divisor(a.N, a.n_mul, a.n_shift);
  // One block takes all heads of its tokens, so that angles are computed once; with few tokens
  // the heads are split over blocks until there are about 8 for every SM. Unsplit and split, us:
  // 8 tokens of 40 heads 34.5 / 9.2, 1000 tokens of 24 heads 26.4 / 13.3, 4000 of 24 18.6 / 19.6
  // (from 32760 on nothing is split).
  const long long split = std::min<long long>((a.heads + 3) / 4, std::max<long long>(1, 1184 / blocks));
  a.per_block = (int)((a.heads + split - 1) / split);
  const dim3 grid((unsigned)blocks, (unsigned)((a.heads + a.per_block - 1) / a.per_block));
  KernelTimer kt(KID_ROTARY, s);
  rotary_kernel<T, V, SPLIT><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

// the widest access that all rows allow: 16 bytes, 8 bytes or single elements (q and k
// [1, 12, 32760, 128] bf16: 77, 83 and 141 us)
template <typename T>
static cudaError_t launch_rotary_t(const RotaryArgs& a, int n, bool half, cudaStream_t s) {
  uint64_t all = (uint64_t)(half ? a.rd / 2 : a.rd) | (uint64_t)(a.d - a.rd);  // in elements
  for (int i = 0; i < n; ++i) {
    all |= reinterpret_cast<uintptr_t>(a.t[i].x) / sizeof(T) | reinterpret_cast<uintptr_t>(a.t[i].y) / sizeof(T);
    for (int j = 0; j < 3; ++j) all |= (uint64_t)a.t[i].xs[j] | (uint64_t)a.t[i].ys[j];
  }
  constexpr int W = 16 / sizeof(T);
  if (all % W == 0) return half ? launch_rotary<T, W, true>(a, half, s) : launch_rotary<T, W, false>(a, half, s);
  if (all % (W / 2) == 0)
    return half ? launch_rotary<T, W / 2, true>(a, half, s) : launch_rotary<T, W / 2, false>(a, half, s);
  return launch_rotary<T, 1, true>(a, half, s);
}

}  // namespace spa2

using namespace spa2;

extern "C" {

spa2_status spa2_rotary(const spa2_rotary_tensor* t, int n, int B, int N, int d, int dtype,
                        const spa2_rotary_spec* spec, int inverse, spa2_stream_t stream) {
  if (!t || !spec || n < 1 || B < 1 || N < 1 || d < 1 || !spec->inv_freq) return SPA2_ERR_INVALID_ARG;
  const int rd = spec->rotary_dim;
  if (n > 2 || d > 1024 || rd < 2 || rd > d || rd % 2 || (long long)B * N > 0x7fffffffLL || spec->axes < 1 ||
      spec->axes > SPA2_ROTARY_MAX_AXES || (dtype != SPA2_DTYPE_BF16 && dtype != SPA2_DTYPE_F32 && dtype != SPA2_DTYPE_F16) ||
      (spec->layout != SPA2_ROTARY_INTERLEAVED && spec->layout != SPA2_ROTARY_HALF))
    return SPA2_ERR_UNSUPPORTED;
  if (spec->positions ? (spec->position_bytes != 4 && spec->position_bytes != 8) : spec->axes != 1)
    return SPA2_ERR_UNSUPPORTED;
  const uintptr_t esz = dtype == SPA2_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(spec->inv_freq) % 8 ||
      (spec->positions && reinterpret_cast<uintptr_t>(spec->positions) % spec->position_bytes))
    return SPA2_ERR_INVALID_ARG;
  RotaryArgs a{};
  a.inv_freq = spec->inv_freq;
  a.scale = spec->scale;
  a.sin_sign = inverse ? -1.f : 1.f;
  a.pos = spec->positions;
  a.pos64 = spec->position_bytes == 8;
  for (int i = 0; i < 3; ++i) a.ps[i] = spec->position_stride[i];
  int pairs = 0;
  for (int i = 0; i < SPA2_ROTARY_MAX_AXES; ++i) {
    a.first[i] = pairs;
    if (i < spec->axes) {
      if (spec->pairs[i] < 0 || spec->pairs[i] > rd / 2) return SPA2_ERR_INVALID_ARG;
      pairs += spec->pairs[i];
    }
  }
  if (pairs != rd / 2) return SPA2_ERR_INVALID_ARG;
  a.tokens = (long long)B * N;
  a.N = N;
  a.d = d;
  a.rd = rd;
  long long heads = 0;
  for (int i = 0; i < n; ++i) {
    if (!t[i].x || !t[i].y || t[i].heads < 1 || reinterpret_cast<uintptr_t>(t[i].x) % esz ||
        reinterpret_cast<uintptr_t>(t[i].y) % esz)
      return SPA2_ERR_INVALID_ARG;
    a.t[i].x = t[i].x;
    a.t[i].y = t[i].y;
    for (int j = 0; j < 3; ++j) {
      a.t[i].xs[j] = t[i].x_stride[j];
      a.t[i].ys[j] = t[i].y_stride[j];
    }
    if (i == 0) a.heads0 = t[i].heads;
    heads += t[i].heads;
  }
  if (heads > 65535) return SPA2_ERR_UNSUPPORTED;
  a.heads = (int)heads;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool half = spec->layout == SPA2_ROTARY_HALF;
  const cudaError_t e = dtype == SPA2_DTYPE_BF16  ? launch_rotary_t<__nv_bfloat16>(a, n, half, s)
                        : dtype == SPA2_DTYPE_F16 ? launch_rotary_t<__half>(a, n, half, s)
                                                  : launch_rotary_t<float>(a, n, half, s);
  return e == cudaSuccess ? SPA2_OK : SPA2_ERR_CUDA;
}

}  // extern "C"
