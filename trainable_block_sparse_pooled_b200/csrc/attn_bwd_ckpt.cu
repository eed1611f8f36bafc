// The dQ pass of the backward on 8-bit checkpoints (spa2_sparse_attn_bwd_ckpt): dQ_i of
// one q-block, and the LSE and D of its rows, which are not kept from the forward and which
// the dK/dV pass then takes from here.
//
// bwd_dq_ckpt_kernel  one CTA per (q-block i, head), two CTAs on an SM. Two passes over the
//   kv-blocks j that i keeps (CSR row of i), with x_ij = scale * log2(e) * (q_i . k_j):
//     first   S = Q K^T, dP = dO V^T;  l = sum_j 2^(x_ij - m), w = sum_j 2^(x_ij - m) dP_ij with
//             a running maximum m, in fp32; then LSE = m + log2 l and D = w / l, for
//             D = rowsum(dO * O) = sum_j P_ij dP_ij. The output O is never formed: no P V
//             product, nothing of its size written or read.
//     second  S and dP again, dS = P * (dP - D), dQ_i += dS K_j * scale.
//   Q_i is decoded from its codes and dO_i scaled on their way into shared memory; K_j and V_j
//   arrive by TMA. The fp16 copies of Q and dO that the dK/dV pass streams are written here too.
//
// Precision: every product takes fp16 operands and adds up in fp32, in this pass as in the dK/dV
// pass. The kept values have 7 bits and are exact in fp16 (a group whose largest magnitude is
// below 4e-6 loses up to 2^-25; above 65504 is clamped and reported). dO is multiplied by a power
// of two that brings the largest |dO| into [4, 8), and on until the largest |dS| that V allows is 2^15 (gradients
// are linear in dO and V: neither the loss's scale nor V's must decide what fp16 leaves of them). With V
// between 4 and 8 that leaves dO's 8 bits exact down to 2^-20 of the largest. Here that is the row's largest, since a row of dQ depends on
// no other row of dO; in the dK/dV pass, whose sums run over the rows, it is the head's. With the head's
// factor alone a row of 2^-12 of the largest would lose 4e-3 of its dQ, one of 2^-16 9e-2. dS, formed in fp32, enters
// dQ = dS K as a pair of halves, 22 bits (bwd_dq_kernel: a pair of bf16). A single half is off by 7e-4 of
// dQ's norm with sink keys of 8x norm, whose terms cancel, and by up to 1.7e-2 in places, of the 2e-2 that is
// promised; the pair by 3e-6 and 1.2e-4 ([12, 8192, 128]). It costs four products a tile, 4% of the step.
//
// What bounds it: each product chain of a CTA is serial (S and dP have one buffer each, dS
// goes over S), so a second CTA on the SM works through its own chain meanwhile, and through
// this one's start and end. That fixes the layout: 256 columns of tensor memory and 113 KB
// of shared memory each, hence Q and dO in shared memory (SS products, bound by the 128
// bytes a cycle that the tensor core reads there), K double-buffered and V single. At
// [12, 32760, 128] with 25.6 of 512 blocks kept: 900 us; the products' shared-memory and tensor
// cycles alone (768 a tile in the first pass, 1280 in the second, 531 tiles an SM) would take 640 us
// at the 1.7 GHz that the power limit leaves. Measured and not kept (with dS as one half): one CTA an SM with Q and dO in
// tensor memory (as bwd_dq_kernel) 1000 us, that with 16 warps 1064; here, Q and dO in tensor memory
// for the first pass 945 against 906, three buffers filled in turn by K and V 914 against 906.
// The forward again for LSE and O (both halves of O stored and read, an fp16 V) took 333 + 34 + 50
// us where the first pass, in bwd_dq_kernel's form, took 390.
//
// It starts while the decoding kernel ends (programmatic dependent launch): the setup, Q_i's codes and
// the lists need nothing of it. The dK/dV pass starts in the same way behind this one.
#include "common.cuh"
#include "kernels.h"

namespace spa2 {

namespace {

constexpr int DQC_THREADS = 320;  // S / dP / dS x 8 warps, TMA, MMA

template <int D>
struct DqcSmem {
  static constexpr int CH = D / 64;
  // Q_i and dO_i fp16; at the end the staged dQ tile (64 KB in fp32 at d = 128)
  alignas(1024) uint8_t q[CH][128 * 128];
  alignas(1024) uint8_t dO[CH][128 * 128];
  alignas(1024) uint8_t k[2][CH][64 * 128];
  alignas(1024) uint8_t v[CH][64 * 128];
  uint64_t q_ready, do_ready;
  uint64_t k_full[2], k_empty[2], v_full, v_empty;
  uint64_t sdp_full, read, ds_full;  // S and dP there; read out; dS there
  uint64_t acc_done, drain;
  uint32_t tmem_base;
  int abort_flag;
  int never;  // stays 0: abort flag of the teardown drains
  uint8_t row_e[128];  // exponent that a row's factor stands for
};
static_assert(2 * (sizeof(DqcSmem<128>) + 1024) <= 228 * 1024, "two CTAs share an SM");

SPA2_DEV bool wait_warp(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
  const bool ok = wait_bar(bar, parity, w);
  return __all_sync(0xffffffff, ok);
}

}  // namespace

// TMEM columns: S 0..63 (over 16 kv columns of it their dS: the high halves in the first 8, the low ones in the
// other 8), dP 64..127, dQ 128 .. 128+d (between the passes: what the two halves of a row exchange).
template <int D, bool TILED>
__global__ void __launch_bounds__(DQC_THREADS, 2)
    bwd_dq_ckpt_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_dq, const __nv_bfloat16* __restrict__ dout,
                       const int8_t* __restrict__ q8, const uint8_t* __restrict__ qe, uint4* __restrict__ q16,
                       uint4* __restrict__ do16, const uint32_t* do_most, float* __restrict__ unscale,
                       float* __restrict__ lse, float* __restrict__ dvec, const int* __restrict__ row_cnt,
                       const int* __restrict__ row_idx,
                       int grad_f32, int N, int Tm, int Tn, float scale, float scale_log2, int* status,
                       unsigned long long wait_limit_ns) {
  constexpr int CH = D / 64;
  constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 64, false, false, /*f16=*/true);
  constexpr uint32_t IDESC_Q = idesc_bf16_f32(128, D, false, true, /*f16=*/true);
  constexpr uint32_t KV_BYTES = 64 * D * 2;
  constexpr uint32_t T_S = 0, T_DP = 64, T_DQ = 128;
  constexpr float LN2 = 0.69314718055994530942f;

  extern __shared__ __align__(1024) uint8_t smem_raw[];  // no room to align it by hand
  DqcSmem<D>& sm = *reinterpret_cast<DqcSmem<D>*>(smem_raw);
  if (smem_u32(smem_raw) & 1023u) {  // the swizzle and the descriptors count on it
    if (threadIdx.x == 0) report(status, SPA2_ERR_CUDA);
    return;
  }

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);  // warp-uniform
  const uint32_t lane = lane_id();
  const int i = blockIdx.x;
  const int bh = blockIdx.y;
  const long long rowid = (long long)bh * Tm + i;

  // what the start waits for, asked for at once: the row's count and first block, and (warps
  // 0-7) Q_i's codes, 16 elements of a row at a time, and dO_i, 8 at a time, neighbours in
  // neighbouring threads
  constexpr int PER_ROW = D / 16, PIECES = 128 * PER_ROW / 256, DO_PIECES = 2 * PIECES;
  const int count = row_cnt[rowid], first = row_idx[rowid * Tn];
  uint4 code[PIECES];
  uint8_t E[PIECES];
  uint4 do_in[DO_PIECES];
  if (warp < 8) {
#pragma unroll
    for (int x = 0; x < PIECES; ++x) {
      const int piece = x * 256 + threadIdx.x, pr = piece / PER_ROW, c = piece % PER_ROW;
      const long long at = (long long)bh * N + (long long)i * 128 + pr;
      const bool there = i * 128 + pr < N;
      code[x] = there ? reinterpret_cast<const uint4*>(q8 + at * D)[c] : make_uint4(0, 0, 0, 0);
      E[x] = there ? qe[at * (D / 32) + (c >> 1)] : (uint8_t)0;
    }
#pragma unroll
    for (int x = 0; x < DO_PIECES; ++x) {
      const int piece = x * 256 + threadIdx.x, pr = piece / (D / 8), c = piece % (D / 8);
      const long long at = (long long)bh * N + (long long)i * 128 + pr;
      do_in[x] = i * 128 + pr < N ? reinterpret_cast<const uint4*>(dout + at * D)[c] : make_uint4(0, 0, 0, 0);
    }
  }

  if (warp == 9) {
    tmem_alloc(&sm.tmem_base, 256);
    tmem_relinquish();
  }
  if (threadIdx.x == 256) {
    mbar_init(&sm.q_ready, 256);
    mbar_init(&sm.do_ready, 256);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    mbar_init(&sm.v_full, 1);
    mbar_init(&sm.v_empty, 1);
    mbar_init(&sm.sdp_full, 1);
    mbar_init(&sm.read, 256);
    mbar_init(&sm.ds_full, 256);
    mbar_init(&sm.acc_done, 1);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    sm.never = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  // Not before this block has its tensor memory: a dK/dV block takes all of an SM's and waits for this grid's
  // end, so it must not come between this block's start and its allocation (by registers the two do not fit
  // on one SM today, by shared memory at d = 64 they would).
  pdl_trigger();
  const WaitCtx wc{&sm.abort_flag, status, wait_limit_ns};
  const WaitCtx drain_wc{&sm.never, nullptr, wait_limit_ns};

  int n = __shfl_sync(0xffffffffu, count, 0);  // warp-uniform
  if (n < 1 || n > Tn) {
    if (threadIdx.x == 0) report(status, SPA2_ERR_DEVICE_BOUNDS);
    n = 0;
  }
  const int* kv_list = row_idx + rowid * Tn;
  int epi_ok = 1;  // a dS thread clears it when its part of the dQ tile was not staged

  if (warp == 8) {
    // ---------------- TMA producer: K and V of 2n tiles ----------------
    if (lane == 0 && n > 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      const int end = 2 * n;
      pdl_wait();  // K and V are decoded by the kernel before
      int kt = 0, vt = 0;  // tiles whose K, whose V has been started
      uint64_t t0 = 0;
      uint32_t idle = 0;
      while (vt < end) {
        // K(kt) needs the products of K(kt - 2) done, V(vt) dP(vt - 1); whichever is free
        if (kt < end && (kt < 2 || mbar_test_wait(&sm.k_empty[kt & 1], ((kt >> 1) - 1) & 1))) {
          const int j = (kt == 0 ? first : kv_list[kt < n ? kt : kt - n]) & TILE_ID_MASK;
          if (j >= Tn) {
            report(status, SPA2_ERR_DEVICE_BOUNDS);
            sm.abort_flag = 1;
            break;
          }
          mbar_expect_tx(&sm.k_full[kt & 1], KV_BYTES);
          for (int c = 0; c < CH; ++c) tma_load_3d(sm.k[kt & 1][c], &tm_k, &sm.k_full[kt & 1], c * 64, j * 64, bh);
          ++kt;
        } else if (vt < kt && (vt < 1 || mbar_test_wait(&sm.v_empty, (vt - 1) & 1))) {
          const int j = (vt == 0 ? first : kv_list[vt < n ? vt : vt - n]) & TILE_ID_MASK;
          mbar_expect_tx(&sm.v_full, KV_BYTES);
          for (int c = 0; c < CH; ++c) tma_load_3d(sm.v[c], &tm_v, &sm.v_full, c * 64, j * 64, bh);
          ++vt;
        } else {
          // nothing free: sleep in try_wait on what frees next, not a hot spin
          if (vt < kt && vt >= 1)
            mbar_try_wait(&sm.v_empty, (vt - 1) & 1);
          else if (kt < end && kt >= 2)
            mbar_try_wait(&sm.k_empty[kt & 1], ((kt >> 1) - 1) & 1);
          if ((++idle & 63u) != 0u) continue;
          if (sm.abort_flag) break;
          const uint64_t now = globaltimer_ns();
          if (t0 == 0) {
            t0 = now;
          } else if (now - t0 > wait_limit_ns) {
            report(status, SPA2_ERR_DEVICE_TIMEOUT);
            sm.abort_flag = 1;
            break;
          }
          continue;
        }
        idle = 0;
        t0 = 0;
      }
      // never leave with copies in flight: wait (bounded) for the last loads
      for (int t = max(0, kt - 2); t < kt; ++t) wait_bar(&sm.k_full[t & 1], (t >> 1) & 1, drain_wc);
      if (vt > 0) wait_bar(&sm.v_full, (vt - 1) & 1, drain_wc);
    }
  } else if (warp == 9) {
    // ---------------- MMA issuer (all 32 lanes; elect.sync picks the issuing lane) ----------------
    if (n > 0) {
      // tile g of the 2n: first pass g < n
      auto issue_s = [&](int g) {
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_el(tmem + T_S, sdesc_sw128(smem_u32(sm.q[kk >> 2]) + (kk & 3) * 32, 16, 1024),
                    sdesc_sw128(smem_u32(sm.k[g & 1][kk >> 2]) + (kk & 3) * 32, 16, 1024), IDESC_S, kk > 0 ? 1u : 0u);
      };
      auto issue_dp = [&]() {
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_el(tmem + T_DP, sdesc_sw128(smem_u32(sm.dO[kk >> 2]) + (kk & 3) * 32, 16, 1024),
                    sdesc_sw128(smem_u32(sm.v[kk >> 2]) + (kk & 3) * 32, 16, 1024), IDESC_S, kk > 0 ? 1u : 0u);
        mma_commit_el(&sm.v_empty);
      };
      // dQ += (dS_hi + dS_lo)(g) K(g), K = 64 kv rows
      auto issue_dq = [&](int g) {
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_el(tmem + T_DQ, tmem + T_S + kk * 8,
                    sdesc_sw128(smem_u32(sm.k[g & 1][0]) + (kk >> 1) * 2048, 64 * 128, 1024), IDESC_Q,
                    (g > n || kk > 0) ? 1u : 0u);
        mma_commit_el(&sm.k_empty[g & 1]);
      };
      bool ok = wait_bar_all(&sm.q_ready, 0, wc);
      // S and dP of the first pass, and of the second one's first tile
      for (int g = 0; g <= n && ok; ++g) {
        ok = wait_bar_all(&sm.k_full[g & 1], (g >> 1) & 1, wc) &&
             (g == 0 || wait_bar_all(&sm.read, (g - 1) & 1, wc));  // the buffers of tile g - 1 are read out
        if (!ok) break;
        issue_s(g);
        if (g < n) mma_commit_el(&sm.k_empty[g & 1]);
        ok = (g > 0 || wait_bar_all(&sm.do_ready, 0, wc)) && wait_bar_all(&sm.v_full, g & 1, wc);
        if (!ok) break;
        issue_dp();
        mma_commit_el(&sm.sdp_full);
      }
      // the rest of the second pass: dP(g) as soon as dP(g - 1) is read out, while dS(g - 1) is
      // still being formed; then dQ(g - 1), and S(g) over its dS
      for (int g = n + 1; g < 2 * n && ok; ++g) {
        ok = wait_bar_all(&sm.v_full, g & 1, wc) && wait_bar_all(&sm.read, (g - 1) & 1, wc);
        if (!ok) break;
        issue_dp();
        ok = wait_bar_all(&sm.ds_full, (g - 1 - n) & 1, wc);
        if (!ok) break;
        issue_dq(g - 1);
        ok = wait_bar_all(&sm.k_full[g & 1], (g >> 1) & 1, wc);
        if (!ok) break;
        issue_s(g);
        mma_commit_el(&sm.sdp_full);
      }
      if (ok && wait_bar_all(&sm.ds_full, (n - 1) & 1, wc)) {
        issue_dq(2 * n - 1);
        mma_commit_el(&sm.acc_done);
      }
      // drain: every MMA issued above completes before TMEM is released
      mma_commit_el(&sm.drain);
      wait_bar_all(&sm.drain, 0, drain_wc);
    }
  } else {
    // ---------------- warps 0-7: warpgroup h handles kv columns 32h .. 32h+31 ----------------
    const int h = warp >> 2;
    const int r = threadIdx.x & 127;  // query row == TMEM lane
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const long long row = (long long)i * 128 + r;
    const bool rvalid = row < N;
    // do_most is written by the kernel before: waited for, and loaded as volatile (the compiler may move
    // a plain load of read-only memory above the wait)
    pdl_wait();
    const uint32_t most = reinterpret_cast<const volatile uint32_t*>(do_most)[(long long)bh * DO_PARTS + lane];
    // Q_i from its codes into shared memory, and its fp16 copy
    bool bad = false;
#pragma unroll
    for (int x = 0; x < PIECES; ++x) {
      const int piece = x * 256 + threadIdx.x, pr = piece / PER_ROW, c = piece % PER_ROW;
      const float step = pack8_step(E[x]);
      const uint32_t in[4] = {code[x].x, code[x].y, code[x].z, code[x].w};
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float f[4];
        pack8_floats(in[e], f);
        // codes of rows behind the last are 0, which the conversion takes for +0
        if (E[x] <= 142) {  // below 2^16: at most 65024
          w[2 * e] = pack_f16(f[0] * step, f[1] * step);
          w[2 * e + 1] = pack_f16(f[2] * step, f[3] * step);
        } else {
          w[2 * e] = pack_f16_clamped(f[0] * step, f[1] * step, bad);
          w[2 * e + 1] = pack_f16_clamped(f[2] * step, f[3] * step, bad);
        }
      }
      const uint4 lo = make_uint4(w[0], w[1], w[2], w[3]), hi = make_uint4(w[4], w[5], w[6], w[7]);
      uint8_t* chunk = sm.q[c >> 2];
      *reinterpret_cast<uint4*>(chunk + sw128_offset(pr, (c & 3) * 2)) = lo;
      *reinterpret_cast<uint4*>(chunk + sw128_offset(pr, (c & 3) * 2 + 1)) = hi;
      if (i * 128 + pr < N) {
        uint4* to = q16 + (((long long)bh * N + (long long)i * 128 + pr) * D + c * 16) / 8;
        to[0] = lo;
        to[1] = hi;
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&sm.q_ready);
    // The power of two that dO is multiplied by. Its exponent field 127 + 129 - E would bring the largest |dO|,
    // 2^(E - 127) or more (of a row for this pass, of the head for the dK/dV pass), into [4, 8); for infinities
    // and NaN, which are reported, and zeros any will do. With |V| < 2^(F - 126), F its largest exponent,
    // |dP - D| < d 2^(F - 122) then: from there it goes down or up until that bound is 2^15, so that dS uses fp16's
    // range and does not leave it whatever the size of V; up by 2^12 at most, where dO itself reaches 2^15.
    const int v_e = (int)__reduce_max_sync(0xffffffffu, most & 0xffffu);
    const int down = max(-12, v_e - 137 + (D == 128 ? 7 : 6));
    auto factor_e = [&](uint32_t e) { return (uint32_t)min(max((int)max(e, 3u) + down, 3), 255); };
    const uint32_t do_e = __reduce_max_sync(0xffffffffu, most) >> 23, most_e = factor_e(do_e);
    const float do_scale = __uint_as_float((256u - most_e) << 23);
    if (i == 0 && threadIdx.x == 0) unscale[bh] = __uint_as_float((most_e - 2u) << 23);  // its inverse
    bad = bad || (int)do_e + down > 255;
    // dO_i to fp16, by its row's factor, and a copy by the head's
#pragma unroll
    for (int x = 0; x < DO_PIECES; ++x) {
      const int piece = x * 256 + threadIdx.x, pr = piece / (D / 8), c = piece % (D / 8);
      const uint4 in = do_in[x];
      uint32_t m = __vmaxu2(__vmaxu2(in.x & 0x7fff7fffu, in.y & 0x7fff7fffu),
                            __vmaxu2(in.z & 0x7fff7fffu, in.w & 0x7fff7fffu));
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int o = 1; o < D / 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t row_e = factor_e(m >> 7);
      if (c == 0) sm.row_e[pr] = (uint8_t)row_e;
      auto to16 = [&](uint32_t w, float by) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
        return do_e <= 254u ? pack_f16(f.x * by, f.y * by)  // below 2^15
                            : pack_f16_clamped(f.x * by, f.y * by, bad);
      };
      auto all16 = [&](float by) { return make_uint4(to16(in.x, by), to16(in.y, by), to16(in.z, by), to16(in.w, by)); };
      *reinterpret_cast<uint4*>(sm.dO[c >> 3] + sw128_offset(pr, c & 7)) =
          all16(__uint_as_float((256u - row_e) << 23));
      if (i * 128 + pr < N) do16[(((long long)bh * N + (long long)i * 128 + pr) * D) / 8 + c] = all16(do_scale);
    }
    fence_proxy_async_smem();
    mbar_arrive(&sm.do_ready);
    if (bad) report(status, SPA2_ERR_RANGE);
    const uint64_t scale2 = f2_pack(scale_log2, scale_log2);
    // only kv-block Tn-1 (last in the ascending list) is ragged
    const int last_valid = (n > 0 && (kv_list[n - 1] & TILE_ID_MASK) == Tn - 1) ? N - (Tn - 1) * 64 : 64;
    bool ok = n > 0;
    // ---- first pass: LSE and D of the row, from its 32 columns of every tile
    float m = -INFINITY, l = 0.f, wsum = 0.f;
    for (int t = 0; t < n && ok; ++t) {
      // a tile excluded for this row's half contributes nothing
      const int kv_valid = (TILED && tile_excluded(kv_list[t], r >> 6)) ? 0 : t == n - 1 ? last_valid : 64;
      if (!wait_warp(&sm.sdp_full, t & 1, wc)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t sa[32], pa[32];
      tmem_ld32(tl + T_S + h * 32, sa);
      tmem_ld32(tl + T_DP + h * 32, pa);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(&sm.read);  // S and dP may be overwritten
      if (kv_valid < 64) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (h * 32 + e >= kv_valid) sa[e] = __float_as_uint(-INFINITY);
      }
      float m4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) m4[e] = __uint_as_float(sa[e]);
#pragma unroll
      for (int e = 4; e < 32; ++e) m4[e & 3] = fmaxf(m4[e & 3], __uint_as_float(sa[e]));
      const float m_new = fmaxf(m, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale_log2);
      if (m_new == -INFINITY) continue;  // nothing kept so far in these columns
      const float alpha = fast_exp2(m - m_new);
      m = m_new;
      const uint64_t neg_m = f2_pack(-m_new, -m_new);
      float l2[2] = {l * alpha, 0.f}, w2[2] = {wsum * alpha, 0.f};
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(sa[2 * e]), __uint_as_float(sa[2 * e + 1])), scale2, neg_m), x0, x1);
        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
        l2[0] += p0;
        l2[1] += p1;
        w2[0] = fmaf(p0, __uint_as_float(pa[2 * e]), w2[0]);
        w2[1] = fmaf(p1, __uint_as_float(pa[2 * e + 1]), w2[1]);
      }
      l = l2[0] + l2[1];
      wsum = w2[0] + w2[1];
    }
    float nlse2 = -INFINITY, Dr = 0.f, back = 0.f;
    if (n > 0) {
      // the two halves of a row meet in the dQ columns, which nothing uses yet
      {
        uint32_t x[16] = {};
        x[0] = __float_as_uint(m);
        x[1] = __float_as_uint(l);
        x[2] = __float_as_uint(wsum);
        tmem_st16(tl + T_DQ + h * 16, x);
        tmem_wait_st();
        tc_fence_before();
        named_bar_sync(1, 256);
        tc_fence_after();
        tmem_ld16(tl + T_DQ + (1 - h) * 16, x);
        tmem_wait_ld();
        const float mo = __uint_as_float(x[0]), M = fmaxf(m, mo);
        if (M > -INFINITY) {
          const float a = fast_exp2(m - M), b = fast_exp2(mo - M);
          // the half of the lower columns first in both threads of the row
          const float l0 = l * a, l1 = __uint_as_float(x[1]) * b, w0 = wsum * a, w1 = __uint_as_float(x[2]) * b;
          l = l0 + l1;
          nlse2 = -(M + log2f(l));
          Dr = (w0 + w1) / l;
        }
      }
      const uint32_t row_e = sm.row_e[r], below = most_e - row_e;
      back = __uint_as_float((row_e - 2u) << 23);
      if (h == 0 && rvalid && ok) {  // +inf: a row that keeps nothing, as the dK/dV pass takes it
        lse[(long long)bh * N + row] = -nlse2 * LN2;
        dvec[(long long)bh * N + row] = below < 127u ? Dr * __uint_as_float((127u - below) << 23) : 0.f;
      }
      if (!rvalid) {
        nlse2 = -INFINITY;
        Dr = 0.f;
      }
      tc_fence_before();  // dQ's first product (after this thread's dS) overwrites those columns
    }
    // ---- second pass: dS
    const uint64_t nlse2x2 = f2_pack(nlse2, nlse2), d2 = f2_pack(Dr, Dr);
    for (int t = 0; t < n && ok; ++t) {
      const int kv_valid = (TILED && tile_excluded(kv_list[t], r >> 6)) ? 0 : t == n - 1 ? last_valid : 64;
      if (!wait_warp(&sm.sdp_full, (n + t) & 1, wc)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t pa[32];
      tmem_ld32(tl + T_DP + h * 32, pa);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(&sm.read);  // dP may be overwritten
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const int c0 = h * 32 + sub * 16;
        uint32_t sa[16], ds[16];
        tmem_ld16(tl + T_S + c0, sa);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sa[2 * e]), __uint_as_float(sa[2 * e + 1])), scale2, nlse2x2), x0, x1);
          float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
          if (kv_valid < 64) {
            if (c0 + 2 * e >= kv_valid) p0 = 0.f;
            if (c0 + 2 * e + 1 >= kv_valid) p1 = 0.f;
          }
          const uint64_t ds2 = f2_mul(
              f2_pack(p0, p1),
              f2_sub(f2_pack(__uint_as_float(pa[sub * 16 + 2 * e]), __uint_as_float(pa[sub * 16 + 2 * e + 1])), d2));
          float s0, s1;
          f2_unpack(ds2, s0, s1);
          ds[e] = pack_f16(s0, s1);
          const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&ds[e]));
          ds[8 + e] = pack_f16(s0 - hi.x, s1 - hi.y);
        }
        tmem_st16(tl + T_S + c0, ds);  // over these columns of S (read by this warp alone)
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.ds_full);
    }
    // epilogue: dQ_i = scale * acc without the row's factor, warpgroup h holding feature columns h*D/2 .. +D/2, staged in
    // the space of Q and dO (every product is done) as 128-byte-swizzled boxes of 128 rows x 128
    // bytes (32 fp32 or 64 bf16 columns) for the TMA stores below; the tensor map clips the rows
    // of a ragged last q-block
    if (ok) ok = wait_warp(&sm.acc_done, 0, wc);
    if (ok) {
      tc_fence_after();
      // scale first: times a far power of two it might be a subnormal number
      auto out = [&](uint32_t acc) { return __uint_as_float(acc) * scale * back; };
      uint8_t* stage = &sm.q[0][0];
#pragma unroll 1
      for (int cc = 0; cc < D / 64; ++cc) {
        const int c0 = h * (D / 2) + cc * 32;  // first feature column of this 32-column slice
        uint32_t a[32];
        tmem_ld32(tl + T_DQ + c0, a);
        tmem_wait_ld();
        if (grad_f32) {
          uint8_t* box = stage + (c0 / 32) * (128 * 128);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(box + sw128_offset(r, e)) =
                make_float4(out(a[4 * e]), out(a[4 * e + 1]),
                            out(a[4 * e + 2]), out(a[4 * e + 3]));
        } else {
          uint8_t* box = stage + (c0 / 64) * (128 * 128);
          const uint32_t u0 = (uint32_t)((c0 % 64) / 8);  // 16-byte unit of the slice in its 64-column box
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(box + sw128_offset(r, u0 + e)) =
                make_uint4(pack_bf16(out(a[8 * e]), out(a[8 * e + 1])),
                           pack_bf16(out(a[8 * e + 2]), out(a[8 * e + 3])),
                           pack_bf16(out(a[8 * e + 4]), out(a[8 * e + 5])),
                           pack_bf16(out(a[8 * e + 6]), out(a[8 * e + 7])));
        }
      }
      fence_proxy_async_smem();
    }
    epi_ok = ok ? 1 : 0;
  }

  tc_fence_before();
  // every thread takes part; the dQ tile is stored only when every dS thread staged its part
  const int all_ok = __syncthreads_and(epi_ok);
  if (threadIdx.x == 0 && all_ok && n > 0) {
    const uint8_t* stage = &sm.q[0][0];
    const int cols = grad_f32 ? 32 : 64;  // columns per 128-byte box
    for (int b = 0; b < D / cols; ++b) tma_store_3d(&tm_dq, stage + b * (128 * 128), b * cols, i * 128, bh);
    tma_store_commit();
    tma_store_wait_all();
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <int D, bool TILED>
static cudaError_t launch_dq_ckpt_t(const BwdArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(DqcSmem<D>);
  const cudaError_t e = cudaFuncSetAttribute(bwd_dq_ckpt_kernel<D, TILED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
  if (e != cudaSuccess) return e;
  KernelTimer kt(KID_BWD_DQ_CKPT, s);
  return launch_k(bwd_dq_ckpt_kernel<D, TILED>, dim3(a.Tm, a.BH), dim3(DQC_THREADS), smem, s, true, *a.tm_k,
                  *a.tm_v, *a.tm_dq, static_cast<const __nv_bfloat16*>(a.dout), a.q8, a.qe, static_cast<uint4*>(a.q16), static_cast<uint4*>(a.do16), a.do_most,
                  a.unscale, a.lse, a.dvec, a.row_cnt, a.row_idx, a.grad_f32, a.N, a.Tm, a.Tn, a.scale, a.scale_log2,
                  a.status, a.wait_limit_ns);
}

cudaError_t launch_dq_ckpt(const BwdArgs& a, int d, cudaStream_t s) {
  if (d == 128) return a.tiled ? launch_dq_ckpt_t<128, true>(a, s) : launch_dq_ckpt_t<128, false>(a, s);
  return a.tiled ? launch_dq_ckpt_t<64, true>(a, s) : launch_dq_ckpt_t<64, false>(a, s);
}

}  // namespace spa2
