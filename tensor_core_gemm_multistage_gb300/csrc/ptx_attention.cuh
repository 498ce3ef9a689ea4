// ptx_attention.cuh - inline-PTX wrappers the masked and tree attention kernels use beside those
// of ptx.cuh: 4-D tensor copies, untiled bulk copies, cluster launch control, bf16 descriptors.
#pragma once

#include "ptx.cuh"

namespace gsr {

// 4-D tiled load global -> shared with an L2 policy (c0 innermost).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
        : "memory");
}

// The same in five dimensions.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3, int32_t c4, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "l"(policy)
        : "memory");
}

// Untiled load global -> shared; addresses 16-byte aligned, `bytes` a multiple of 16.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Cluster launch control: asks to take over a CTA of this grid that has not started.  The 16-byte
// answer lands at `dst` and counts on `bar`.
__device__ __forceinline__ void clc_try_cancel(uint32_t dst, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
                 "r"(bar)
                 : "memory");
}
// The x index of the CTA taken over, or -1: none is left (and none may be asked for again).
__device__ __forceinline__ int clc_taken(uint32_t src) {
    int x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "mov.s32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
        : "=r"(x)
        : "r"(src)
        : "memory");
    return x;
}

// Moves registers between warpgroups: every warp of one gives registers back (dec) or takes them (inc,
// which waits until they are there).  The shares times 128 threads stay within what the CTA was
// launched with.
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 64 bytes of one thread to global memory: whole 32-byte sectors in two instructions where the address
// allows it, else in four of 16 bytes.
__device__ __forceinline__ void store_64_bytes(void* to, const uint32_t (&v)[16]) {
    if ((reinterpret_cast<uintptr_t>(to) & 31u) == 0u) {
#pragma unroll
        for (int i = 0; i < 16; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<uint32_t*>(to) + i),
                         "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]),
                         "r"(v[i + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<uint4*>(static_cast<uint32_t*>(to) + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

// Programmatic dependent launch: waits until the launches this one depends on have finished and their
// writes are visible; lets the next one's CTAs start once every CTA has come here (or ended).
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Instruction descriptor as idesc_f16_f32, for f16 (0) or bf16 (1) operands, both of one type.
__host__ __device__ constexpr uint32_t idesc_16_f32(bool bf16, int M, int N, bool a_mn_major, bool b_mn_major) {
    return idesc_f16_f32(M, N, a_mn_major, b_mn_major) | (bf16 ? (1u << 7) | (1u << 10) : 0u);
}

}  // namespace gsr
