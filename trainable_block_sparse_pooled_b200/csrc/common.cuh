// Device helpers shared by the spa2 kernels: inline-PTX wrappers for mbarriers,
// TMA (cp.async.bulk.tensor), tcgen05 (TMEM alloc / MMA / ld / st / commit),
// bounded waits that report a timeout through a device status word instead of
// hanging, and the shared-memory matrix / instruction descriptors used by the
// tcgen05 MMAs. Written for sm_100a only.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spa2.h"

#define SPA2_DEV __device__ __forceinline__

namespace spa2 {

// ---------------------------------------------------------------------------
// status word: the first 4 bytes of every workspace; kernels only move it away
// from SPA2_OK (first error wins), the host reads it with spa2_stream_status.
// ---------------------------------------------------------------------------
SPA2_DEV void report(int* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

SPA2_DEV uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

SPA2_DEV uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

SPA2_DEV uint32_t lane_id() { return threadIdx.x & 31; }
SPA2_DEV uint32_t warp_id() { return __shfl_sync(0xffffffff, threadIdx.x >> 5, 0); }

SPA2_DEV bool elect_one() {
  uint32_t pred = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

// ---------------------------------------------------------------------------
// mbarrier
// ---------------------------------------------------------------------------
SPA2_DEV void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

SPA2_DEV void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

SPA2_DEV void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

SPA2_DEV void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

SPA2_DEV bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// non-blocking probe: has the phase of the given parity completed?
SPA2_DEV bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Per-CTA abort flag + time limit. A wait that runs past the limit records
// SPA2_ERR_DEVICE_TIMEOUT, raises the CTA's abort flag and returns false; every
// other wait in the CTA then gives up at once, so the CTA reaches its teardown
// (TMEM release) instead of spinning forever.
struct WaitCtx {
  volatile int* abort_flag;  // in shared memory
  int* status;               // global status word
  uint64_t limit_ns;
};

SPA2_DEV bool wait_bar(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
  if (mbar_try_wait(bar, parity)) return true;
  // try_wait suspends the thread for a while when the phase is open, so polling it
  // is cheap; the abort flag and the clock (a special-register read that would
  // compete with exp2 for issue) are looked at only every 64 polls
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 63u) == 0u) {
      if (*w.abort_flag) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) {
        t0 = t;
      } else if (t - t0 > w.limit_ns) {
        report(w.status, SPA2_ERR_DEVICE_TIMEOUT);
        *w.abort_flag = 1;
        return false;
      }
    }
  }
}

// Waits for a warp that issues with the *_el calls: every lane waits (and so
// takes the acquire itself); the result is true only when every lane saw the
// phase, which keeps the caller's control flow warp-uniform.
SPA2_DEV bool wait_bar_all(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
  const bool ok = wait_bar(bar, parity, w);
  return __all_sync(0xffffffffu, ok);
}

SPA2_DEV bool test_wait_all(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_test_wait(bar, parity));
}

// ---------------------------------------------------------------------------
// TMA (tiled, no multicast)
// ---------------------------------------------------------------------------
SPA2_DEV void tma_prefetch_desc(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

SPA2_DEV void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// L2 prefetch of one box of a tiled tensor (no shared memory, no barrier)
SPA2_DEV void tma_prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// untiled bulk copy global -> shared (16-byte aligned addresses, size multiple of 16)
SPA2_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

SPA2_DEV void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

SPA2_DEV void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
SPA2_DEV void tma_store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 16-byte global -> shared copy through L2 only; src_bytes = 0 writes zeros
SPA2_DEV void cp_async16(void* dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(src_bytes)
               : "memory");
}
SPA2_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
SPA2_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

SPA2_DEV int ld_acquire_gpu(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

SPA2_DEV void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

SPA2_DEV void named_bar_sync(int id, int nthreads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// ---------------------------------------------------------------------------
// tcgen05: tensor memory and 5th-generation tensor-core MMA
// ---------------------------------------------------------------------------
SPA2_DEV void tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {  // whole warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
}
SPA2_DEV void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
SPA2_DEV void tmem_dealloc(uint32_t taddr, uint32_t ncols) {  // whole warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
SPA2_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
SPA2_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D[tmem] (+)= A[smem] * B[smem]
SPA2_DEV void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]
SPA2_DEV void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ---------------------------------------------------------------------------
// Warp-wide issue of tensor-core work. tcgen05.mma and tcgen05.commit act once
// per executing thread. An issue loop run by a single lane keeps its operand
// descriptors off the warp-uniform datapath and was measured to issue one
// 128x64x16 product per ~70 cycles, where the tensor core finishes one in 48
// (the 128 B/cycle it reads from shared memory); run by all 32 lanes, with
// elect.sync choosing the lane that issues, the same loop keeps the tensor core
// busy. Every lane must reach these calls together, so the caller keeps the
// control flow around them warp-uniform (wait_bar_all / test_wait_all).
SPA2_DEV void mma_ss_el(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

SPA2_DEV void mma_ts_el(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

SPA2_DEV void mma_commit_el(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// arrive once on `bar` when every tcgen05 op issued so far by this thread is done
SPA2_DEV void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// 32 lanes x 32 consecutive 32-bit columns; thread i of the warp gets lane (base lane + i)
SPA2_DEV void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// 32 lanes x 16 consecutive 32-bit columns
SPA2_DEV void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 32 lanes x 64 consecutive 32-bit columns
SPA2_DEV void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
        "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
        "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr));
}

SPA2_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

SPA2_DEV void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

SPA2_DEV void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
SPA2_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle, sm_100 layout (version 1).
// lbo / sbo in bytes. For K-major operands sbo is the stride between 8-row
// groups (1024 B for 128-byte rows) and lbo is unused; for MN-major operands
// lbo is the stride between 64-element MN chunks and sbo the stride between
// 8-row K groups.
SPA2_DEV uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;  // descriptor version for sm_100
  d |= 2ull << 61;  // SWIZZLE_128B
  return d;
}

// Instruction descriptor of kind::f16 with fp32 accumulation; A and B are both
// bf16 (default) or both fp16 (f16 = true).
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, bool a_mn_major, bool b_mn_major,
                                                      bool f16 = false) {
  return (1u << 4)                                // D format: f32
         | ((f16 ? 0u : 1u) << 7)                 // A format: f16 = 0, bf16 = 1
         | ((f16 ? 0u : 1u) << 10)                // B format: f16 = 0, bf16 = 1
         | ((a_mn_major ? 1u : 0u) << 15)         // A major
         | ((b_mn_major ? 1u : 0u) << 16)         // B major
         | (static_cast<uint32_t>(N >> 3) << 17)  // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24); // M / 16
}

// byte offset of 16-byte unit `u` of row `r` in a 128-byte-swizzled tile (tile base 1024-aligned)
SPA2_DEV uint32_t sw128_offset(uint32_t r, uint32_t u) { return r * 128u + ((u ^ (r & 7u)) << 4); }

SPA2_DEV uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);  // .x = lo (low 16 bits), .y = hi
  return *reinterpret_cast<uint32_t*>(&v);
}

SPA2_DEV uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);  // .x = lo (low 16 bits), .y = hi
  return *reinterpret_cast<uint32_t*>(&v);
}

// ---------------------------------------------------------------------------
// Programmatic dependent launch. A kernel launched with launch_k(..., pdl =
// true) may start while the previous kernel of its stream is still running;
// it calls pdl_wait() before it reads anything that kernel (or earlier work)
// wrote and may do independent work before. pdl_trigger() lets the next
// PDL-launched kernel start early. The first kernel of every C-ABI call is
// launched without the attribute, so it is ordered after whatever the caller
// enqueued before the call; only the call's later kernels use it.
// ---------------------------------------------------------------------------
SPA2_DEV void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
SPA2_DEV void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Params, typename... Args>
static inline cudaError_t launch_k(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                   bool pdl, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// packed fp32 pairs (sm_100 f32x2 arithmetic): low half = first element
SPA2_DEV uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(__float_as_uint(lo)), "r"(__float_as_uint(hi)));
  return r;
}
SPA2_DEV void f2_unpack(uint64_t v, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  lo = __uint_as_float(a);
  hi = __uint_as_float(b);
}
SPA2_DEV uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
SPA2_DEV uint64_t f2_sub(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
SPA2_DEV uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// ---------------------------------------------------------------------------
// Tile lists. The attention kernels work on tiles of 128 query rows x 64 key
// rows and read, per query tile (forward, dQ) or key tile (dK/dV), a list of
// the tiles it meets. An entry is a tile id in bits 0-29; bit 30 (31) set
// means rows 0-63 (64-127) of the 128-row query tile are excluded from it,
// which happens when 64-row query blocks share a tile but keep different
// key blocks. With 128-row query blocks and 64-row key blocks the block CSR /
// CSC are the tile lists as they are (no bit set).
// ---------------------------------------------------------------------------
constexpr int TILE_ID_MASK = 0x3FFFFFFF;
SPA2_DEV bool tile_excluded(int entry, int half) { return ((unsigned)entry >> (30 + half)) & 1u; }

// ---------------------------------------------------------------------------
// 8-bit groups (spa2_pack8). E is the biased fp32 exponent field of a group's
// largest magnitude, so x * 2^(127 - E) lies in (-2, 2) and a code counts steps of
// 2^(E - 133), 1/64 of that unit.
// ---------------------------------------------------------------------------
// 2^(127 - E); E = 254 needs an fp32 subnormal, which products here keep. For E =
// 255 the codes do not matter.
SPA2_DEV float pack8_scale(uint32_t E) { return __uint_as_float(E < 254u ? (254u - E) << 23 : 0x00400000u); }
// rint(64 x scale) clamped to +-127: x scale is exact wherever it can reach a code
// other than 0, and adding 1.5 * 2^23 rounds to the nearest integer, ties to even,
// and leaves it in the low bits
SPA2_DEV int8_t pack8_code(float x, float scale) {
  const float y = fminf(fmaxf(x * scale, -1.984375f), 1.984375f);
  return (int8_t)(__float_as_uint(fmaf(y, 64.f, 12582912.f)) & 0xffu);
}
// the same of two values, as 16-bit integers, where scale64 = 64 * pack8_scale(E) is a
// finite normal number (7 <= E <= 254): one product, clamped after the rounding
SPA2_DEV uint32_t pack8_code2(float a, float b, float scale64) {
  const uint32_t two = __byte_perm(__float_as_uint(fmaf(a, scale64, 12582912.f)),
                                   __float_as_uint(fmaf(b, scale64, 12582912.f)), 0x5410);
  return __vmins2(__vmaxs2(two, 0xff81ff81u), 0x007f007fu);
}
// the four codes of w as floats: a code plus 128 in the low bits of 2^23 is 2^23 + 128 + code
SPA2_DEV void pack8_floats(uint32_t w, float (&f)[4]) {
  w ^= 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | i)) - 8388736.f;
}
// 2^(E - 133), below E = 7 an fp32 subnormal; NaN for E = 255
SPA2_DEV float pack8_step(uint32_t E) {
  return __uint_as_float(E >= 255u ? 0x7fffffffu : E >= 7u ? (E - 6u) << 23 : 1u << (16u + E));
}

// (a, b) as an fp16 pair; |x| > 65504 (or NaN) is clamped and flagged
SPA2_DEV uint32_t pack_f16_clamped(float a, float b, bool& bad) {
  if (!(fabsf(a) <= 65504.f) || !(fabsf(b) <= 65504.f)) {
    bad = true;
    a = fminf(fmaxf(a, -65504.f), 65504.f);
    b = fminf(fmaxf(b, -65504.f), 65504.f);
  }
  return pack_f16(a, b);
}

SPA2_DEV float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One head's kv columns (Tn counts from head * Tn on), longest first, written
// as global column indices head * Tn + c: a counting sort by one 256-thread
// block (keys clamped to [0, 1023]; the order among equal counts is whatever the
// shared-memory atomics give, which does not matter: a column's gradients are
// computed the same way whichever CTA takes it and whenever). The persistent
// dK/dV pass takes its columns head by head and, within a head, long columns
// first: it does not end on a long column, and the Q / dO tiles the running
// columns share stay within one head's worth of L2.
// early > 0: the `early` longest columns of every head come before all others (rank by
// rank), so that a column that most query blocks keep (attention sinks) does not start when the
// rest is nearly done. Of these the first `ranks` (of equal columns the lower ones: whether a column
// is taken in parts decides how its sums are rounded, so it must not depend on the atomics) are
// listed `parts` times, for the parts of their tiles: order has heads * (Tn + ranks * (parts - 1))
// entries.
constexpr int MAX_RANKS = 4;
SPA2_DEV void longest_first(const int* __restrict__ cnt, int Tn, int head, int* __restrict__ order, int heads = 0,
                            int early = 0, int ranks = 0, int parts = 1) {
  constexpr int KEYS = 1024, PER = KEYS / 256;
  __shared__ int start[KEYS];
  __shared__ int warp_sum[8];
  __shared__ unsigned long long warp_most[8];
  __shared__ int chosen[MAX_RANKS];
  const int t = threadIdx.x;
  const int* cnt_h = cnt + (long long)head * Tn;
  const int more = ranks * (parts - 1);  // entries of a head beyond one per column
  int* out_h = order + (long long)(early + more) * heads + (long long)head * (Tn - early) - early;
  auto is_chosen = [&](int c, int n) {
    bool is = false;
    for (int x = 0; x < n; ++x) is = is || chosen[x] == c;
    return is;
  };
  for (int rank = 0; rank < ranks; ++rank) {  // ranks <= Tn: there is one left
    unsigned long long most = 0;
    for (int c = t; c < Tn; c += 256)
      if (!is_chosen(c, rank))
        most = max(most, (unsigned long long)(min(max(cnt_h[c], 0), KEYS - 1) + 1) << 32 | (0xffffffffu - (uint32_t)c));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    if ((t & 31) == 0) warp_most[t >> 5] = most;
    __syncthreads();
    if (t == 0) {
      for (int w = 1; w < 8; ++w) most = max(most, warp_most[w]);
      const int c = (int)(0xffffffffu - (uint32_t)most);
      chosen[rank] = c;
      for (int x = 0; x < parts; ++x) order[(long long)(rank * parts + x) * heads + head] = head * Tn + c;
    }
    __syncthreads();
  }
  for (int k = t; k < KEYS; k += 256) start[k] = 0;
  __syncthreads();
  for (int c = t; c < Tn; c += 256)
    if (!is_chosen(c, ranks)) atomicAdd(&start[min(max(cnt_h[c], 0), KEYS - 1)], 1);
  __syncthreads();
  // exclusive scan in descending key order: thread t owns keys KEYS-1-PER*t ... KEYS-PER-PER*t
  int bin[PER], sum = 0;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    bin[e] = start[KEYS - 1 - PER * t - e];
    sum += bin[e];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if ((t & 31) >= o) incl += y;
  }
  if ((t & 31) == 31) warp_sum[t >> 5] = incl;
  __syncthreads();
  int base = incl - sum;
  for (int w = 0; w < (t >> 5); ++w) base += warp_sum[w];
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    start[KEYS - 1 - PER * t - e] = base;
    base += bin[e];
  }
  __syncthreads();
  for (int c = t; c < Tn; c += 256) {
    if (is_chosen(c, ranks)) continue;
    const int rank = ranks + atomicAdd(&start[min(max(cnt_h[c], 0), KEYS - 1)], 1);
    (rank < early ? order[(long long)(rank + more) * heads + head] : out_h[rank]) = head * Tn + c;
  }
  __syncthreads();  // start[] is reused by the next head of this block
}

}  // namespace spa2
