// Activation checkpoints in 8 bits (spa2_pack8 / spa2_unpack8 in
// include/spa2.h): groups of 32 elements of a row share one exponent byte E, the
// biased fp32 exponent of their largest magnitude; code = rint(x * 2^(133 - E)),
// value = code * 2^(E - 133).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace spa2 {

namespace {

struct Pack8Args {
  spa2_pack8_tensor t[SPA2_PACK8_MAX];
};

}  // namespace

// one warp per group, one lane per element
template <typename T>
__global__ void __launch_bounds__(256) pack8_kernel(const Pack8Args a) {
  const spa2_pack8_tensor& t = a.t[blockIdx.y];
  const long long per_row = (t.d + 31) / 32, groups = t.rows * per_row;
  for (long long g = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); g < groups; g += (long long)gridDim.x * 8) {
    const long long row = g / per_row, e = (g % per_row) * 32 + lane_id();
    const float x = e < t.d ? static_cast<float>(static_cast<const T*>(t.x)[row * t.d + e]) : 0.f;
    const uint32_t E = __reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7fffffffu) >> 23;
    if (e < t.d) t.codes[row * t.d + e] = pack8_code(x, pack8_scale(E));
    if (lane_id() == 0) t.exps[g] = (uint8_t)E;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) unpack8_kernel(const Pack8Args a) {
  const spa2_pack8_tensor& t = a.t[blockIdx.y];
  const long long per_row = (t.d + 31) / 32, groups = t.rows * per_row;
  for (long long g = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); g < groups; g += (long long)gridDim.x * 8) {
    const long long row = g / per_row, e = (g % per_row) * 32 + lane_id();
    const float step = pack8_step(t.exps[g]);
    if (e < t.d) static_cast<T*>(t.x)[row * t.d + e] = static_cast<T>(static_cast<float>(t.codes[row * t.d + e]) * step);
  }
}

template <typename T>
static cudaError_t launch_pack8_t(const Pack8Args& a, int n, bool unpack, cudaStream_t s) {
  long long groups = 0;
  for (int i = 0; i < n; ++i) groups = std::max(groups, (long long)(a.t[i].rows * ((a.t[i].d + 31) / 32)));
  if (groups == 0) return cudaSuccess;
  const dim3 grid((unsigned)std::min((groups + 7) / 8, 1LL << 20), (unsigned)n);
  KernelTimer kt(unpack ? KID_UNPACK8 : KID_PACK8, s);
  if (unpack)
    unpack8_kernel<T><<<grid, 256, 0, s>>>(a);
  else
    pack8_kernel<T><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pack8(const spa2_pack8_tensor* t, int n, int dtype, bool unpack, cudaStream_t s) {
  Pack8Args a{};
  for (int i = 0; i < n; ++i) a.t[i] = t[i];
  return dtype == SPA2_DTYPE_BF16  ? launch_pack8_t<__nv_bfloat16>(a, n, unpack, s)
         : dtype == SPA2_DTYPE_F16 ? launch_pack8_t<__half>(a, n, unpack, s)
                                   : launch_pack8_t<float>(a, n, unpack, s);
}

static spa2_status pack8_call(const spa2_pack8_tensor* t, int n, int dtype, bool unpack, spa2_stream_t stream) {
  if (!t || n < 1) return SPA2_ERR_INVALID_ARG;
  if (n > SPA2_PACK8_MAX || (dtype != SPA2_DTYPE_BF16 && dtype != SPA2_DTYPE_F32 && dtype != SPA2_DTYPE_F16))
    return SPA2_ERR_UNSUPPORTED;
  const uintptr_t esz = dtype == SPA2_DTYPE_F32 ? 4 : 2;
  for (int i = 0; i < n; ++i) {
    if (t[i].rows < 0 || t[i].d < 1) return SPA2_ERR_INVALID_ARG;
    if (t[i].rows > (1LL << 40) / t[i].d) return SPA2_ERR_UNSUPPORTED;
    if (t[i].rows && (!t[i].x || !t[i].codes || !t[i].exps || reinterpret_cast<uintptr_t>(t[i].x) % esz))
      return SPA2_ERR_INVALID_ARG;
  }
  return launch_pack8(t, n, dtype, unpack, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SPA2_OK
                                                                                                 : SPA2_ERR_CUDA;
}

}  // namespace spa2

using namespace spa2;

extern "C" {

spa2_status spa2_pack8(const spa2_pack8_tensor* t, int n, int dtype, spa2_stream_t stream) {
  return pack8_call(t, n, dtype, false, stream);
}

spa2_status spa2_unpack8(const spa2_pack8_tensor* t, int n, int dtype, spa2_stream_t stream) {
  return pack8_call(t, n, dtype, true, stream);
}

}  // extern "C"
