// Device helpers shared by the attention kernels: 16-bit packing, bounded waits
// on mbarriers, the TMA boxes of a paged cache, tcgen05 descriptors.
#pragma once

#include "pkv_common.cuh"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr int kStageTokens = 16;      // tokens of a TMA box of the cache (and of a decode stage)
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per wait before giving up

// Context length of sequence b as the kernels use it: negative or too long
// values are clamped (and flagged by the decode kernel).
__device__ __forceinline__ int clamped_len(int n, int cap) { return n < 0 ? 0 : (n > cap ? cap : n); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack2(uint32_t x, __nv_bfloat16) {
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&x));
}
__device__ __forceinline__ float2 unpack2(uint32_t x, __half) {
    return __half22float2(*reinterpret_cast<__half2*>(&x));
}

// 16-token box of K or V for KV head g at token offset toff of block blk,
// 64-dim region starting at dim c0, in either cache layout.
__device__ __forceinline__ void load_kv_box(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int g, int toff, int blk, bool hnd,
                                            uint64_t policy) {
    if (hnd)
        ptx::tma_load_4d(dst, map, bar, c0, toff, g, blk, policy);
    else
        ptx::tma_load_4d(dst, map, bar, c0, g, toff, blk, policy);
}

// Bounded wait on an mbarrier phase.  Returns false (after raising the CTA's
// abort flag and the device error bit on expiry) if the phase did not complete.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           int32_t* err_flag,
                                           uint64_t limit_ns = kWaitLimitNs) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (true) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (ptx::globaltimer() - t0 > limit_ns) {
            *abort_flag = 1;
            flag_error(err_flag, PKV_EFLAG_TIMEOUT);
            return false;
        }
    }
}

#ifdef PKV_DEBUG
// Debug builds (-DPKV_DEBUG) fill ring slots with all-ones bytes, a NaN in
// fp16, bf16 and E4M3 alike, whenever their contents stop being valid: the
// whole ring at the start, and each slot when its stage is released.  A read
// of a slot whose copy has not landed, or of a stage already released, then
// turns the output to NaN instead of passing unnoticed.  `lanes` threads
// (lane index `lane`) share the fill; each makes its writes visible to the
// async proxy, which writes the slot next.
__device__ __forceinline__ void poison_smem(uint8_t* base, int bytes, int lane, int lanes) {
    for (int i = lane; i < bytes / 16; i += lanes)
        reinterpret_cast<uint4*>(base)[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
    ptx::fence_proxy_async_smem();
}
#endif

// Instruction descriptor of tcgen05.mma kind::f16: fp32 accumulator, A and B
// of one 16-bit type (0 = fp16, 1 = bf16), A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t mma_idesc(uint32_t fmt, int m, int n, bool b_mn_major) {
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
template <typename T> struct F16Format;
template <> struct F16Format<__half> { static constexpr uint32_t value = 0; };
template <> struct F16Format<__nv_bfloat16> { static constexpr uint32_t value = 1; };

// A bounded wait whose outcome is the same for the whole warp (a lane that
// gives up raises the CTA's abort flag; the warp then leaves together, so
// warp-collective tensor-memory instructions never run on part of a warp).
__device__ __forceinline__ bool warp_wait_phase(uint32_t bar, uint32_t parity,
                                                volatile int* abort_flag, int32_t* err_flag) {
    const bool ok = wait_phase(bar, parity, abort_flag, err_flag);
    return __all_sync(0xffffffffu, ok);
}

// Two fp32 weights as hi + lo 16-bit terms packed in pairs (element 0 in the
// low half).  bf16: both terms by truncation (a bit mask; hi + lo keeps p to
// 2^-14 relative); fp16: both terms rounded to nearest.
__device__ __forceinline__ void split_hi_lo(float p0, float p1, uint32_t& hi, uint32_t& lo,
                                            __nv_bfloat16) {
    const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
    hi = __byte_perm(b0, b1, 0x7632);
    const float r0 = p0 - __uint_as_float(b0 & 0xffff0000u);
    const float r1 = p1 - __uint_as_float(b1 & 0xffff0000u);
    lo = __byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x7632);
}
__device__ __forceinline__ void split_hi_lo(float p0, float p1, uint32_t& hi, uint32_t& lo, __half) {
    hi = pack2(p0, p1, __half());
    const float2 back = unpack2(hi, __half());
    lo = pack2(p0 - back.x, p1 - back.y, __half());
}

}  // namespace pkv
