// Rotary positions (spa2_rotary in include/spa2.h): pairs of a head's row turned
// by position * frequency, forward (angle theta) and backward (angle -theta).
//
// rotary_kernel  one thread per (token, pair or copied element) and head.
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
};

template <typename T>
SPA2_DEV float to_f32(T x) { return static_cast<float>(x); }
template <typename T>
SPA2_DEV T from_f32(float x) { return static_cast<T>(x); }
template <>
SPA2_DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
SPA2_DEV __half from_f32<__half>(float x) { return __float2half_rn(x); }

// cos and sin of position * inv_freq[p], both times the scale. The angle is
// counted in turns and reduced to [-1/2, 1/2] in fp64 (a far position times a
// frequency has more whole turns than fp32 has digits), then taken in fp32.
SPA2_DEV float2 cos_sin(const RotaryArgs& a, long long token, int p) {
  const long long b = token / a.N, n = token % a.N;
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

}  // namespace

template <typename T, bool HALF>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryArgs a) {
  const int units = a.rd / 2 + (a.d - a.rd);
  const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
  if (idx >= a.tokens * units) return;
  const long long token = idx / units;
  const int u = (int)(idx % units);
  const long long b = token / a.N, n = token % a.N;
  int h = blockIdx.y;
  const RotaryTensor& t = a.t[h >= a.heads0];
  if (h >= a.heads0) h -= a.heads0;
  const T* x = static_cast<const T*>(t.x) + b * t.xs[0] + h * t.xs[1] + n * t.xs[2];
  T* y = static_cast<T*>(t.y) + b * t.ys[0] + h * t.ys[1] + n * t.ys[2];
  if (u >= a.rd / 2) {
    const int e = a.rd + u - a.rd / 2;
    y[e] = x[e];
    return;
  }
  const int i = HALF ? u : 2 * u, j = HALF ? u + a.rd / 2 : 2 * u + 1;
  const float2 cs = cos_sin(a, token, u);
  const float v = to_f32(x[i]), w = to_f32(x[j]);
  y[i] = from_f32<T>(v * cs.x - w * cs.y);
  y[j] = from_f32<T>(v * cs.y + w * cs.x);
}

template <typename T>
static cudaError_t launch_rotary(const RotaryArgs& a, int layout, cudaStream_t s) {
  const long long threads = a.tokens * (a.rd / 2 + (a.d - a.rd));
  const long long blocks = (threads + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, (unsigned)a.heads);
  KernelTimer kt(KID_ROTARY, s);
  if (layout == SPA2_ROTARY_HALF)
    rotary_kernel<T, true><<<grid, 256, 0, s>>>(a);
  else
    rotary_kernel<T, false><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
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
  const cudaError_t e = dtype == SPA2_DTYPE_BF16  ? launch_rotary<__nv_bfloat16>(a, spec->layout, s)
                        : dtype == SPA2_DTYPE_F16 ? launch_rotary<__half>(a, spec->layout, s)
                                                  : launch_rotary<float>(a, spec->layout, s);
  return e == cudaSuccess ? SPA2_OK : SPA2_ERR_CUDA;
}

}  // extern "C"
