// PTX wrappers that only the 8-bit products use: block-scaled tcgen05 MMAs, the
// copy of their scales into tensor memory, untiled bulk copies, and the
// kernels' bounded waits. Written against the PTX ISA.
#pragma once

#include "ptx.cuh"

namespace mmbwd {
namespace q8 {

// Untiled bulk copy global -> this CTA's shared memory, completing on `bar`
// (16-byte aligned addresses, size a multiple of 16).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// 32 rows of 16 bytes (512 contiguous bytes of shared memory: 8-row groups of
// 128 bytes) into four tensor-memory columns, repeated in all four lane
// quadrants. Pair form: each CTA of the pair copies from its own shared memory
// into its own tensor memory, at the same addresses.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128u >> 4) << 32) | (1ull << 46);
}
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns: thread i receives lane (taddr.lane + i).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Instruction descriptor of kind::mxf8f6f4 with ue8m0 scales, K-major operands:
// A and B format at bits 7-9 and 10-12 (0 e4m3, 1 e5m2), N >> 3 at 17-22, the
// scale type (1: ue8m0) at 23, M >> 4 at 24-28; which byte of a scale word an
// MMA takes, of B at 4-5 and of A at 29-30 (scale_id).
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N, int a_format, int b_format) {
    return (static_cast<uint32_t>(a_format) << 7) | (static_cast<uint32_t>(b_format) << 10) |
           (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t scale_id(uint32_t id) { return (id << 4) | (id << 29); }

// D[tmem] (+)= (A . scale A) . (B . scale B)^T over 32 values of K, one scale per
// row and instruction, scales in tensor memory; one elected thread.
__device__ __forceinline__ void mma_mxf8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                              uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}
__device__ __forceinline__ void mma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}

// 32 contiguous bytes between registers and global memory. `left`: elements up to
// the row's end (none is touched beyond it), `per16`: elements in 16 bytes, `wide`:
// what every row's start is a multiple of, and with it the rows' length: 32 bytes
// (2), 16 (1) or 8 (0).
__device__ __forceinline__ void st256(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void st256(void* p, const uint32_t* v, int64_t left, int per16, int wide) {
    if (wide == 2) {
        if (left > 0) st256(p, v);
    } else if (wide == 1) {
        uint4* q = static_cast<uint4*>(p);
        if (left > 0) q[0] = make_uint4(v[0], v[1], v[2], v[3]);
        if (left > per16) q[1] = make_uint4(v[4], v[5], v[6], v[7]);
    } else {
        uint2* q = static_cast<uint2*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (left > i * per16 / 2) q[i] = make_uint2(v[2 * i], v[2 * i + 1]);
    }
}
__device__ __forceinline__ void ld256(const void* p, uint32_t* v, int64_t left, int per16, int wide) {
    if (wide == 2) {
        if (left > 0)
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                         : "l"(p)
                         : "memory");
    } else if (wide == 1) {
        const uint4* q = static_cast<const uint4*>(p);
        if (left > 0) {
            const uint4 a = q[0];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        }
        if (left > per16) {
            const uint4 a = q[1];
            v[4] = a.x, v[5] = a.y, v[6] = a.z, v[7] = a.w;
        }
    } else {
        const uint2* q = static_cast<const uint2*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (left > i * per16 / 2) {
                const uint2 a = q[i];
                v[2 * i] = a.x, v[2 * i + 1] = a.y;
            }
    }
}

constexpr unsigned long long TEARDOWN_NS = 2000000000ull;  // teardown waits, whatever the limit of the others

// Where a wait gave up (device status word of the 8-bit products).
enum Site : int { SITE_EMPTY = 1, SITE_ACC_FREE = 2, SITE_FULL = 3, SITE_ACC_FULL = 4, SITE_TEARDOWN = 8, SITE_SELFTEST = 9, SITE_FORWARD = 10 };

// Bounded mbarrier wait: false after `limit_ns` (recorded in `status`) or once
// another warp of the CTA has given up. A teardown wait ignores the latter, and
// lasts up to TEARDOWN_NS however short the limit: copies and MMAs in flight have
// to land before their memory goes.
struct Waiter {
    volatile uint32_t* abort;
    unsigned int* status;
    unsigned long long limit_ns;

    __device__ void record(int site, int item) const {
        *abort = 1u;
        if (atomicCAS(&status[0], 0u, static_cast<unsigned>(-MMBWD_ERR_DEVICE_TIMEOUT)) == 0u) {
            status[1] = blockIdx.x;
            status[2] = static_cast<unsigned>(site);
            status[3] = static_cast<unsigned>(item);
            __threadfence();
        }
    }
    __device__ bool wait(uint32_t bar, uint32_t parity, int site, int item, bool teardown = false) const {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = ptx::globaltimer(), limit = teardown ? TEARDOWN_NS : limit_ns;
        for (uint32_t i = 1;; ++i) {
            if (ptx::mbar_try_wait(bar, parity)) return true;
            if ((i & 31u) == 0) {
                if (!teardown && *abort) return false;
                if (ptx::globaltimer() - t0 > limit) {
                    record(site, item);
                    return false;
                }
            }
        }
    }
    __device__ bool wait_warp(uint32_t bar, uint32_t parity, int site, int item) const {
        const bool ok = wait(bar, parity, site, item);
        return __all_sync(0xffffffffu, ok);
    }
};

// The body of each kernel's wait self-test (one thread): nothing ever arrives on
// the barrier, so the wait has to give up and record it.
__device__ __forceinline__ void selftest_wait(unsigned int* status, unsigned long long limit_ns) {
    __shared__ alignas(8) uint64_t bar;
    __shared__ uint32_t abort_flag;
    abort_flag = 0u;
    ptx::mbar_init(ptx::smem_u32(&bar), 1u);
    ptx::fence_mbar_init();
    Waiter{&abort_flag, status, limit_ns}.wait(ptx::smem_u32(&bar), 0u, SITE_SELFTEST, 0);
}

}  // namespace q8
}  // namespace mmbwd
