// Activation checkpoints in 8 bits (spa2_pack8 / spa2_unpack8 in
// include/spa2.h): groups of 32 elements of a row share one exponent byte E, the
// biased fp32 exponent of their largest magnitude; code = rint(x * 2^(133 - E)),
// value = code * 2^(E - 133).
//
// Both kernels move bytes and little else (bf16: 3 + 1/32 bytes per element): bound by HBM. Eight
// elements of a row are a chunk (one 16-byte access, two for fp32), four chunks a
// group; a thread takes UNROLL chunks, 256 apart, and loads them all before it works on the
// first, so that enough of them are in flight to cover HBM's latency. The group's largest
// exponent meets over two shuffles. Measured, four tensors [393120, 128] bf16 (610 MB each way):
// pack 94 us, unpack 88 us = 6.5 and 6.9 TB/s with the 126 MB that L2 still holds of the last
// pass, 0.94 of the measured copy rate over both; UNROLL 4 against 1, 2, 8: 100 + 92 us (from cold
// L2) against 124 + 113, 111 + 95, 125 + 108. A ragged fp16 tensor [32760, 1000] 23 + 17 us, for
// 15 us of bytes each: two microseconds of start, and blocks in 7 waves.
// Where tensors fit in L2 the instructions count as well: a code costs a conversion, a fused
// multiply-add and half a clamp of a 16-bit pair, its value a byte permutation, an addition and a
// product (no integer conversions, which run at a quarter of the rate).
// pack8_kernel, unpack8_kernel                rows that 16-byte accesses fit
// pack8_single_kernel, unpack8_single_kernel  any others: one lane per element (ten times slower:
//                                             1033 + 1006 us on the tensors above)
// unpack8_step_kernel                         what the attention's backward starts from
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace spa2 {

namespace {

struct Pack8Args {
  spa2_pack8_tensor t[SPA2_PACK8_MAX];
  uint32_t* f16[SPA2_PACK8_MAX];        // packing: fp16 copy of the tensor, or null
  int* status;                          // where |x| > 65504 is reported; needed for a copy
  uint32_t per_row[SPA2_PACK8_MAX];     // chunk places of a row, and x / per_row = x * div_mul >> (32 + div_shift)
  uint32_t div_mul[SPA2_PACK8_MAX], div_shift[SPA2_PACK8_MAX];  // for x < 2^31
};

constexpr int CHUNK = 8, PER_GROUP = 4, UNROLL = 4, THREADS = 256;
constexpr int PLACES = UNROLL * THREADS;  // chunk places of a block
constexpr int EARLY_COLUMNS = 8;          // a head's columns that the dK/dV pass takes before all others

template <typename T>
struct alignas(16) Chunk {
  T e[CHUNK];
};

// The chunk places of a tensor are numbered row by row, whole groups to a row, so that the
// last group of a row may hold places without a chunk. One thread's places of a block:
template <bool FLAT>
struct Places {
  uint32_t per_row, mul, shift, first;
  long long row0, base;

  SPA2_DEV Places(const Pack8Args& a) {
    base = (long long)blockIdx.x * PLACES;
    if (!FLAT) {
      per_row = a.per_row[blockIdx.y];
      mul = a.div_mul[blockIdx.y];
      shift = a.div_shift[blockIdx.y];
      row0 = base / per_row;
      first = (uint32_t)(base - row0 * per_row);
    }
  }
  // first element and group of place c (0 .. PLACES - 1); false where there is no chunk
  SPA2_DEV bool at(const spa2_pack8_tensor& t, uint32_t c, long long& e, long long& group) const {
    if (FLAT) {  // every row is whole groups
      e = (base + c) * CHUNK;
      group = (base + c) / PER_GROUP;
      return e < t.rows * t.d;
    }
    const uint32_t p = first + c, r = __umulhi(p, mul) >> shift, col = p - r * per_row;
    const long long row = row0 + r;
    e = row * t.d + (long long)col * CHUNK;
    group = row * (per_row / PER_GROUP) + col / PER_GROUP;
    return row < t.rows && (long long)col * CHUNK < t.d;
  }
};

SPA2_DEV float value_of(uint32_t bits, __nv_bfloat16) { return __uint_as_float(bits << 16); }
SPA2_DEV float value_of(uint32_t bits, __half) { return __half2float(__ushort_as_half((unsigned short)bits)); }

// largest magnitude's fp32 exponent field over a chunk, NaN and infinities being the largest
template <typename T>
SPA2_DEV uint32_t chunk_exponent(const Chunk<T>& x) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
  if constexpr (sizeof(T) == 2) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    return __float_as_uint(value_of(m, T())) >> 23;  // m has no sign
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) m = max(m, w[i] & 0x7fffffffu);
    return m >> 23;
  }
}

// fp16 copy of a chunk of a bf16 tensor or of kept values, whose largest has the exponent E; below
// 2^16 (E <= 142) these are at most 65280 and no element needs a look
SPA2_DEV void store_f16(uint32_t* to, const float (&f)[CHUNK], uint32_t E, bool& bad) {
  uint4 w;
  if (E <= 142u)
    w = make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
  else
    w = make_uint4(pack_f16_clamped(f[0], f[1], bad), pack_f16_clamped(f[2], f[3], bad),
                   pack_f16_clamped(f[4], f[5], bad), pack_f16_clamped(f[6], f[7], bad));
  *reinterpret_cast<uint4*>(to) = w;
}

}  // namespace

// FLAT, rows of whole groups, needs no division: 100 + 92 us against 117 + 102 on the tensors above.
// There six blocks to an SM (40 registers) gain 3%; with ragged rows they would cost 20%, and fp32
// chunks would spill.
template <typename T, bool FLAT>
__global__ void __launch_bounds__(THREADS, FLAT && sizeof(T) == 2 ? 6 : 1)
    pack8_kernel(const __grid_constant__ Pack8Args a) {
  pdl_trigger();
  const spa2_pack8_tensor& t = a.t[blockIdx.y];
  const Places<FLAT> places(a);
  uint32_t* f16 = a.f16[blockIdx.y];
  long long e[UNROLL], group[UNROLL];
  bool here[UNROLL], bad = false;
  Chunk<T> x[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    here[u] = places.at(t, u * THREADS + threadIdx.x, e[u], group[u]);
    x[u] = Chunk<T>{};
    if (here[u]) x[u] = *reinterpret_cast<const Chunk<T>*>(static_cast<const T*>(t.x) + e[u]);
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    uint32_t E = chunk_exponent(x[u]);
    E = max(E, __shfl_xor_sync(0xffffffffu, E, 1));
    E = max(E, __shfl_xor_sync(0xffffffffu, E, 2));
    if (!here[u]) continue;
    float f[CHUNK];
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) f[i] = static_cast<float>(x[u].e[i]);
    uint32_t c[4];  // codes as 16-bit integers
    if (E - 7u < 248u) {
      const float scale64 = __uint_as_float((260u - E) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = pack8_code2(f[2 * i], f[2 * i + 1], scale64);
    } else {  // magnitudes below 2^-120, or a group whose codes do not matter
      const float scale = pack8_scale(E);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = __byte_perm((int)pack8_code(f[2 * i], scale), (int)pack8_code(f[2 * i + 1], scale), 0x5410);
    }
    *reinterpret_cast<uint2*>(t.codes + e[u]) =
        make_uint2(__byte_perm(c[0], c[1], 0x6420), __byte_perm(c[2], c[3], 0x6420));
    if (threadIdx.x % PER_GROUP == 0) t.exps[group[u]] = (uint8_t)E;
    if (f16) store_f16(f16 + e[u] / 2, f, E, bad);
  }
  if (bad) report(a.status, SPA2_ERR_RANGE);
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(THREADS, FLAT && sizeof(T) == 2 ? 6 : 1)
    unpack8_kernel(const __grid_constant__ Pack8Args a) {
  const spa2_pack8_tensor& t = a.t[blockIdx.y];
  const Places<FLAT> places(a);
  long long e[UNROLL], group;
  bool here[UNROLL];
  uint2 code[UNROLL];
  uint8_t E[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    here[u] = places.at(t, u * THREADS + threadIdx.x, e[u], group);
    if (here[u]) {
      code[u] = *reinterpret_cast<const uint2*>(t.codes + e[u]);
      E[u] = t.exps[group];
    }
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    if (!here[u]) continue;
    const float step = pack8_step(E[u]);
    float lo[4], hi[4];
    pack8_floats(code[u].x, lo);
    pack8_floats(code[u].y, hi);
    Chunk<T> x;
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) x.e[i] = static_cast<T>((i < 4 ? lo[i & 3] : hi[i & 3]) * step);
    *reinterpret_cast<Chunk<T>*>(static_cast<T*>(t.x) + e[u]) = x;
  }
}

// one warp per group, one lane per element
template <typename T>
__global__ void __launch_bounds__(THREADS) pack8_single_kernel(const __grid_constant__ Pack8Args a) {
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
__global__ void __launch_bounds__(THREADS) unpack8_single_kernel(const __grid_constant__ Pack8Args a) {
  const spa2_pack8_tensor& t = a.t[blockIdx.y];
  const long long per_row = (t.d + 31) / 32, groups = t.rows * per_row;
  for (long long g = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); g < groups; g += (long long)gridDim.x * 8) {
    const long long row = g / per_row, e = (g % per_row) * 32 + lane_id();
    const float step = pack8_step(t.exps[g]);
    if (e < t.d) static_cast<T*>(t.x)[row * t.d + e] = static_cast<T>(static_cast<float>(t.codes[row * t.d + e]) * step);
  }
}

template <typename T>
static cudaError_t launch_pack8_t(Pack8Args& a, int n, bool unpack, cudaStream_t s) {  // n >= 1 tensors, none empty
  long long groups = 0;
  bool chunks = true, flat = true;
  for (int i = 0; i < n; ++i) {
    const spa2_pack8_tensor& t = a.t[i];
    groups = std::max(groups, (long long)(t.rows * ((t.d + 31) / 32)));
    chunks &= t.d % CHUNK == 0 && t.d < (1LL << 31) && reinterpret_cast<uintptr_t>(t.x) % 16 == 0 &&
              reinterpret_cast<uintptr_t>(t.codes) % CHUNK == 0;
    flat &= t.d % SPA2_PACK8_GROUP == 0;
    // x / p = x * ceil(2^(31 + l) / p) >> (31 + l) for x < 2^31, with 2^l >= p the next power of two
    const uint64_t p = (uint64_t)((t.d + 31) / 32 * PER_GROUP);
    if (chunks) {
      uint32_t l = 0;
      while ((1ull << l) < p) ++l;
      a.per_row[i] = (uint32_t)p;
      a.div_mul[i] = (uint32_t)(((1ull << (31 + l)) + p - 1) / p);
      a.div_shift[i] = l - 1;
    }
  }
  KernelTimer kt(unpack ? KID_UNPACK8 : KID_PACK8, s);
  if (chunks) {
    const dim3 grid((unsigned)((groups * PER_GROUP + PLACES - 1) / PLACES), (unsigned)n);
    auto* k = unpack ? (flat ? unpack8_kernel<T, true> : unpack8_kernel<T, false>)
                     : (flat ? pack8_kernel<T, true> : pack8_kernel<T, false>);
    k<<<grid, THREADS, 0, s>>>(a);
  } else {
    const dim3 grid((unsigned)std::min((groups + 7) / 8, 1LL << 20), (unsigned)n);
    (unpack ? unpack8_single_kernel<T> : pack8_single_kernel<T>)<<<grid, THREADS, 0, s>>>(a);
  }
  return cudaGetLastError();
}

static cudaError_t launch(Pack8Args& a, int n, int dtype, bool unpack, cudaStream_t s) {
  return dtype == SPA2_DTYPE_BF16  ? launch_pack8_t<__nv_bfloat16>(a, n, unpack, s)
         : dtype == SPA2_DTYPE_F16 ? launch_pack8_t<__half>(a, n, unpack, s)
                                   : launch_pack8_t<float>(a, n, unpack, s);
}

cudaError_t launch_pack8_step(const spa2_pack8_tensor (&t)[3], void* v16, int* status, cudaStream_t s) {
  Pack8Args a{};
  std::copy(t, t + 3, a.t);
  a.f16[2] = static_cast<uint32_t*>(v16);
  a.status = status;
  return launch(a, 3, SPA2_DTYPE_BF16, false, s);
}

// What the backward on checkpoints starts from, by the row of the grid: 0 the largest |dO| of every
// head and the largest exponent of V in the blocks that a query keeps, in DO_PARTS parts, 1 the order
// in which the dK/dV pass takes its columns, 2, 3 the kept values of K and V as fp16 (exact where a
// group's largest is between 4e-6 and 65504; beyond, clamped, and reported by the dK/dV pass if a
// query keeps them). The few blocks of the first two rows work longest and start first (last, they
// would end 15 us after the others). 63 us at [12, 32760, 128], for 404 MB: the measured copy rate.
__global__ void __launch_bounds__(THREADS, 6) unpack8_step_kernel(const __grid_constant__ Unpack8Step a) {
  pdl_trigger();
  if (blockIdx.y == 1) {
    for (int head = blockIdx.x; head < a.heads; head += gridDim.x) {
      longest_first(a.col_cnt, a.Tn, head, a.col_order, (int)a.heads, min(a.Tn, EARLY_COLUMNS), a.split.ranks,
                    a.split.parts);
      if (threadIdx.x < a.split.ranks * 4) a.split.done[(threadIdx.x / 4 * a.heads + head) * 4 + threadIdx.x % 4] = 0;
    }
    return;
  }
  if (blockIdx.y == 0) {
    __shared__ uint32_t most[THREADS / 32], v_most[THREADS / 32];
    const long long chunks = a.per_head / CHUNK;
    const int per_row = a.d / 32;  // exponents of a row: 2 or 4
    for (int item = blockIdx.x; item < a.heads * DO_PARTS; item += gridDim.x) {
      const int head = item / DO_PARTS, part = item % DO_PARTS;
      const uint4* x = static_cast<const uint4*>(a.dout) + head * chunks;
      uint32_t m = 0;
#pragma unroll 8
      for (long long c = part * chunks / DO_PARTS + threadIdx.x; c < (part + 1) * chunks / DO_PARTS; c += THREADS) {
        const uint4 w = x[c];
        m = __vmaxu2(__vmaxu2(m, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu);
        m = __vmaxu2(__vmaxu2(m, w.z & 0x7fff7fffu), w.w & 0x7fff7fffu);
      }
      m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
      uint32_t e = 0;
      for (long long row = (long long)part * a.N / DO_PARTS + threadIdx.x; row < (long long)(part + 1) * a.N / DO_PARTS;
           row += THREADS) {
        if (a.col_cnt[(long long)head * a.Tn + row / 64] <= 0) continue;
        const uint8_t* x = a.v.exps + ((long long)head * a.N + row) * per_row;
        for (int i = 0; i < per_row; ++i) e = max(e, x[i] <= 142 ? (uint32_t)x[i] : 0u);  // above: clamped
      }
      e = __reduce_max_sync(0xffffffffu, e);
      if (lane_id() == 0) {
        most[threadIdx.x / 32] = m;
        v_most[threadIdx.x / 32] = e;
      }
      __syncthreads();
      if (threadIdx.x < 32) {
        m = __reduce_max_sync(0xffffffffu, threadIdx.x < THREADS / 32 ? most[threadIdx.x] : 0u);
        e = __reduce_max_sync(0xffffffffu, threadIdx.x < THREADS / 32 ? v_most[threadIdx.x] : 0u);
        if (threadIdx.x == 0) a.do_most[item] = m << 16 | e;  // fp32 bits of |dO|, the exponent below them
      }
      __syncthreads();
    }
    return;
  }
  const bool second = blockIdx.y == 3;
  const int8_t* codes = second ? a.v.codes : a.k.codes;
  const uint8_t* exps = second ? a.v.exps : a.k.exps;
  uint32_t* out = second ? a.v16 : a.k16;
  const long long end = a.heads * a.per_head / CHUNK, base = (long long)blockIdx.x * PLACES + threadIdx.x;
  uint2 code[UNROLL];
  uint8_t E[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const long long c = base + u * THREADS;
    if (c < end) {
      code[u] = reinterpret_cast<const uint2*>(codes)[c];
      E[u] = exps[c / PER_GROUP];
    }
  }
  bool clamped = false;
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const long long c = base + u * THREADS;
    if (c >= end) continue;
    const float step = pack8_step(E[u]);
    float lo[4], hi[4], f[CHUNK];
    pack8_floats(code[u].x, lo);
    pack8_floats(code[u].y, hi);
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) f[i] = (i < 4 ? lo[i & 3] : hi[i & 3]) * step;
    store_f16(out + c * (CHUNK / 2), f, E[u], clamped);
  }
}

cudaError_t launch_unpack8_step(const Unpack8Step& a, cudaStream_t s) {
  const long long chunks = a.heads * a.per_head / CHUNK;
  KernelTimer kt(KID_UNPACK8, s);
  // short sequences: a block for each part of a head, up to four an SM (17 us with 8 blocks for 64 parts)
  const long long blocks = std::max((chunks + PLACES - 1) / PLACES, std::min(a.heads * DO_PARTS, 592LL));
  unpack8_step_kernel<<<dim3((unsigned)blocks, 4), THREADS, 0, s>>>(a);
  return cudaGetLastError();
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
  // without the empty ones, for which the kernels' division by places per row has no divisor
  Pack8Args a{};
  const int full = (int)(std::copy_if(t, t + n, a.t, [](const spa2_pack8_tensor& x) { return x.rows > 0; }) - a.t);
  if (full == 0) return SPA2_OK;
  return launch(a, full, dtype, unpack, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SPA2_OK : SPA2_ERR_CUDA;
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
