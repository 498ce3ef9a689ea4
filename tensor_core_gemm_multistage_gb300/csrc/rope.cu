// rope.cu - norms of queries and keys for each head with the position rotation in the same pass, its
// gradient, and the writes of keys and values to a paged cache of 16 or 4 bits with both on the way.
//
// A row x of D values becomes rot(n w), n = x / sqrt(mean(x^2) + eps): pair (a, b) of the first R columns
// turns to (a c - b s, b c + a s).  Every row is read and written once and carries a few operations a byte,
// so the time is that of the bytes (4 D a row forwards, 6 D backwards), or of the launch.
//
// A row is held by D / 16 lanes in two 16-byte pieces each, chosen so that a lane has both halves of its
// pairs: nothing but the sums crosses lanes.  A warp takes consecutive steps of 512 / D rows, a token's heads after
// one another, so that the token's angles are loaded once into registers (for each row, they would be twice the
// row's bytes).  Rows come through a ring in shared memory, several steps ahead (cp.async, each lane its own pieces,
// so that no lane waits for another): plain loads ahead would take the registers that the arithmetic needs.  So two
// CTAs of 256 threads an SM, all of them there from the start, keep two or three steps of each warp on the way.
//
// Measured, bf16, D = 128, norm and rotation: 8192 tokens of 40 heads 31 us (5.6 TB/s, 83 % of a large copy's rate; a copy of these
// 84 MB takes 26), the gradient 50 us (5.1 TB/s); 48 tokens of 48 heads into pages 3.1 us.  What is between is issue
// (61 and 54 % of the slots, a warp's arithmetic in a row): fewer instructions made each step, f32x2 forms the most.
#include "rows16.cuh"
#include "serving.h"

namespace gsr {
namespace {

// Five CTAs of 128 threads with 102 registers take as long forwards, and spill in the gradient (72 us for 50) and the writes.
constexpr int kThreads = 256, kWarps = kThreads / 32, kCtasAnSm = 2;

// ---------------------------------------------------------------------------
// Two floats in a register pair: one instruction works on both
// ---------------------------------------------------------------------------
typedef unsigned long long f2;
__device__ __forceinline__ f2 two(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f2 both(float x) { return two(x, x); }
__device__ __forceinline__ float2 parts_of(f2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum_of(f2 x) {
    const float2 f = parts_of(x);
    return f.x + f.y;
}

// ---------------------------------------------------------------------------
// A lane's part of a row
// ---------------------------------------------------------------------------
// 16-byte pieces c0 and c1, neighbouring lanes' next to each other (a warp's access then covers whole sectors; with
// both of a lane's pieces next to each other a plain copy took 44 us for 26).
struct LanePart {
    int c0, c1;
    bool t0, t1;                 // interleaved: whether a piece's pairs turn; else (t0) whether they turn with each other
};
template <int LANES, bool INTERLEAVED>
__device__ __forceinline__ LanePart lane_part(int l, int R) {
    const int rc = R >> 4;                       // lanes that hold pairs (i, i + R / 2)
    if (INTERLEAVED) return {l, l + LANES, 8 * l < R, 8 * (l + LANES) < R};
    if (l < rc) return {l, l + rc, true, true};
    return {l + rc, l + LANES, false, false};
}
// 16 values: v[0..3] are piece c0, v[4..7] piece c1.
template <class T>
__device__ __forceinline__ void unpack_part(const uint4& lo, const uint4& hi, f2 (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = Pair<T>::unpack((&lo.x)[i]), y = Pair<T>::unpack((&hi.x)[i]);
        v[i] = two(x.x, x.y);
        v[4 + i] = two(y.x, y.y);
    }
}
template <class T>
__device__ __forceinline__ uint4 pack_piece(const f2* v) {
    uint4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = parts_of(v[i]);
        (&r.x)[i] = Pair<T>::pack(x.x, x.y);
    }
    return r;
}
template <class T>
__device__ __forceinline__ void load_weight(const void* w, const LanePart& at, f2 (&to)[8]) {
    unpack_part<T>(__ldg(static_cast<const uint4*>(w) + at.c0), __ldg(static_cast<const uint4*>(w) + at.c1), to);
}
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ---------------------------------------------------------------------------
// Rotation
// ---------------------------------------------------------------------------
struct Angles {
    f2 c[4], s[4];               // cosines and sines of a lane's eight pairs
};
// BACK: turned the other way.
template <bool BACK, int LANES, bool INTERLEAVED>
__device__ __forceinline__ void load_angles(Angles& a, const float* row, int R, const LanePart& at, int l) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (!(i ? at.t1 : at.t0)) continue;
        const float* c = row + (INTERLEAVED ? 4 * (l + i * LANES) : 8 * l + 4 * i);
        const float4 x = __ldg(reinterpret_cast<const float4*>(c)), y = __ldg(reinterpret_cast<const float4*>(c + R / 2));
        a.c[2 * i] = two(x.x, x.y);
        a.c[2 * i + 1] = two(x.z, x.w);
        a.s[2 * i] = BACK ? two(-y.x, -y.y) : two(y.x, y.y);
        a.s[2 * i + 1] = BACK ? two(-y.z, -y.w) : two(y.z, y.w);
    }
}
// (a, b) -> (a c - b s, b c + a s).  EXACT: each product and sum rounded by itself, so that codes of 4 bits do not
// hang on a contraction.
template <bool EXACT, bool INTERLEAVED>
__device__ __forceinline__ void rotate(f2 (&v)[8], const Angles& a, const LanePart& at) {
    if (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!(i < 4 ? at.t0 : at.t1)) continue;
            const float2 x = parts_of(v[i]), cc = parts_of(a.c[i / 2]), ss = parts_of(a.s[i / 2]);
            const float c = i & 1 ? cc.y : cc.x, s = i & 1 ? ss.y : ss.x;
            if (EXACT) v[i] = two(__fsub_rn(__fmul_rn(x.x, c), __fmul_rn(x.y, s)), __fadd_rn(__fmul_rn(x.y, c), __fmul_rn(x.x, s)));
            else v[i] = two(fmaf(x.x, c, -x.y * s), fmaf(x.y, c, x.x * s));
        }
    } else if (at.t0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f2 x = v[i], y = v[4 + i];
            if (EXACT) {                                   // (products and sums of pairs come out contracted)
                const float2 f = parts_of(x), g = parts_of(y), c = parts_of(a.c[i]), t = parts_of(a.s[i]);
                v[i] = two(__fsub_rn(__fmul_rn(f.x, c.x), __fmul_rn(g.x, t.x)), __fsub_rn(__fmul_rn(f.y, c.y), __fmul_rn(g.y, t.y)));
                v[4 + i] = two(__fadd_rn(__fmul_rn(g.x, c.x), __fmul_rn(f.x, t.x)), __fadd_rn(__fmul_rn(g.y, c.y), __fmul_rn(f.y, t.y)));
            } else {
                const float2 t = parts_of(a.s[i]);
                v[i] = fma2(y, two(-t.x, -t.y), mul2(x, a.c[i]));
                v[4 + i] = fma2(x, a.s[i], mul2(y, a.c[i]));
            }
        }
    }
}
// The angles of one token after another.
struct TokenAngles {
    Angles angles;
    int token = -1, pos = 0, next_pos = 0;
    bool known = true;                  // the position is in the table
    template <bool BACK, int LANES, bool INTERLEAVED>
    __device__ __forceinline__ void move(const RopeParams& p, int now, int s, const LanePart& at, int l) {
        if (now == token || !p.table) return;
        if (p.positions) {
            pos = now == token + 1 && token >= 0 ? next_pos : __ldg(p.positions + now);
            next_pos = now + 1 < p.B * p.S ? __ldg(p.positions + now + 1) : 0;
        } else {
            pos = s;
        }
        token = now;
        known = pos >= 0 && pos < p.rows;
        if (known) load_angles<BACK, LANES, INTERLEAVED>(angles, p.table + (long long)pos * p.R, p.R, at, l);
    }
};

// ---------------------------------------------------------------------------
// A warp's steps, and the ring that its rows come through
// ---------------------------------------------------------------------------
// A step is as many rows of one token as a warp holds: of Q's heads, then of K's (cache writes: and as many of V's).
struct RopePlan {
    Divider by_token, by_seq, by_page;
    int q_steps, k_steps, units;        // steps of a token's two parts; all steps
};
struct Walk {
    int left;                           // steps that have not been opened
    int token, b, s, part, done;        // the token and its batch row and place; its part, and the steps of it so far
    int run, h0;                        // steps left of the open run, and its first row's head
    // Steps [w each, w each + each) of all, for warp w of `warps`.
    __device__ __forceinline__ Walk(const RopePlan& plan, int w, int warps) {
        const int each = (plan.units + warps - 1) / warps;
        const int first = (int)min((long long)w * each, (long long)plan.units);
        left = min(each, plan.units - first);
        token = plan.by_token(first);
        done = first - token * (int)plan.by_token.d;
        part = done >= plan.q_steps;
        if (part) done -= plan.q_steps;
        b = plan.by_seq(token);
        s = token - b * (int)plan.by_seq.d;
        run = h0 = 0;
    }
    // The next run of steps of one token's part; `left` is above 0.
    __device__ __forceinline__ void open(const RopePlan& plan, int rows) {
        while (done >= (part ? plan.k_steps : plan.q_steps)) {
            done = 0;
            part ^= 1;
            if (part) continue;
            ++token;
            if (++s == (int)plan.by_seq.d) {
                s = 0;
                ++b;
            }
        }
        run = min((part ? plan.k_steps : plan.q_steps) - done, left);
        h0 = done * rows;
        done += run;
        left -= run;
    }
};

__device__ __forceinline__ void copy_piece(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint4 ring_piece(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
// By value: a chosen reference to a kernel's parameter is read through memory.
__device__ __forceinline__ Strided pick(bool first, const Strided& a, const Strided& b) {
    return {first ? a.data : b.data, first ? a.batch : b.batch, first ? a.head : b.head, first ? a.row : b.row};
}
// N streams of rows (the same heads of the same tokens), STAGES steps of them; each lane copies and reads its own pieces.
template <int N, int STAGES>
struct Ring {
    static constexpr uint32_t STAGE = N * 2 * 512;
    uint32_t base, to, at;              // of this lane: the ring, the stage that is copied next, the one that is read next
    Walk ahead;
    const char* from[N];                // the lane's next row in each stream, null without one
    long long step[N];                  // bytes to the next step's row
    int next[N], live;                  // bytes to the lane's second piece; heads from the lane's on
    __device__ __forceinline__ Ring(void* smem, int lane, const Walk& w)
        : base((uint32_t)__cvta_generic_to_shared(smem) + 16 * lane), to(base), at(base), ahead(w), live(0) {}
    __device__ __forceinline__ uint32_t after(uint32_t stage) const { return stage == base + (STAGES - 1) * STAGE ? base : stage + STAGE; }
    // rows(part, n, &at): stream n's operand and pieces, without data where it has none; heads(part).
    template <int ROWS, class Rows, class Heads>
    __device__ __forceinline__ void load(const RopePlan& plan, int row, Rows rows, Heads heads) {
        if (ahead.run == 0 && ahead.left > 0) {
            ahead.open(plan, ROWS);
            const int h = ahead.h0 + row;
            live = heads(ahead.part) - h;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                LanePart part;
                const Strided src = rows(ahead.part, n, part);
                from[n] = src.data ? static_cast<const char*>(src.data) + 2 * (ahead.b * src.batch + ahead.s * src.row + h * src.head) + 16 * part.c0
                                   : nullptr;
                next[n] = 16 * (part.c1 - part.c0);
                step[n] = src.data ? 2 * ROWS * src.head : 0;
            }
        }
        if (ahead.run > 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (live > 0 && from[n]) {
                    copy_piece(to + n * 1024, from[n]);
                    copy_piece(to + n * 1024 + 512, from[n] + next[n]);
                }
                from[n] += step[n];
            }
            live -= ROWS;
            --ahead.run;
            to = after(to);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // After a load: the pieces of the step that is read next are there.
    __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory"); }
    __device__ __forceinline__ void read(int n, uint4& lo, uint4& hi) const {
        lo = ring_piece(at + n * 1024);
        hi = ring_piece(at + n * 1024 + 512);
    }
    __device__ __forceinline__ void advance() { at = after(at); }
};

// ---------------------------------------------------------------------------
// Rows of 4 bits
// ---------------------------------------------------------------------------
// Of three values; the larger is NaN where one of them is.
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void ends_of(const f2* v, float& low, float& high) {
    const float2 a = parts_of(v[0]), b = parts_of(v[1]), c = parts_of(v[2]), d = parts_of(v[3]);
    low = min3(min3(a.x, a.y, b.x), min3(b.y, c.x, c.y), fminf(d.x, d.y));
    high = max3(max3(a.x, a.y, b.x), max3(b.y, c.x, c.y), max3(d.x, d.y, d.y));
}
// Eight codes of values v, scale s and minimum m as held.
__device__ __forceinline__ uint32_t codes_of(const f2* v, float s, float m) {
    uint32_t w = 0u;
    if (!(s > 0.0f)) return w;
    // (v - m) / s as 15 times what a saturated product leaves in 0..1, off by less than 2^-16 (1 + |m| / 15 s): divided
    // only next to a border.  A sum with 1.5 2^23 rounds to the nearest even and leaves the integer in its low bits
    // (conversions run at an eighth of the rate).
    constexpr uint32_t MAGIC = 0x4b400000u;
    const float magic = __uint_as_float(MAGIC), inv = __fdividef(1.0f, 15.0f * s), shift = -m * inv;
    const f2 fifteen = both(15.0f), above = both(magic), below = both(-magic);
    float worst = 0.0f;                                     // distance from an integer: a border is at a half
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = parts_of(v[i]);
        const f2 y = two(__saturatef(fmaf(x.x, inv, shift)), __saturatef(fmaf(x.y, inv, shift))), c = fma2(y, fifteen, above);
        const float2 a = parts_of(c), off = parts_of(fma2(y, both(-15.0f), add2(c, below)));
        worst = max3(worst, fabsf(off.x), fabsf(off.y));
        w += __float_as_uint(a.x) * (1u << (8 * i)) + __float_as_uint(a.y) * (16u << (8 * i));
    }
    if (s > 1e-30f && s < 1e30f && worst < 0.5f - 0x1p-16f - 0x1p-16f * fabsf(shift)) return w - MAGIC * 0x11111111u;
    w = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = parts_of(v[i]);
        w |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(x.x - m, s)), 0.0f), 15.0f) << (8 * i);
        w |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(x.y - m, s)), 0.0f), 15.0f) << (8 * i + 4);
    }
    return w;
}
// These writes follow the number of instructions, minimum, maximum and codes of every value on top of the rotation: 24576
// tokens of 8 x 128 with K's rotation 51 us (129 MB, 2.5 TB/s). No unit is full (64 % of the issue slots, 48 % of the integer
// pipe): two CTAs of 128 registers an SM do not cover a warp's own latencies.
//
// Per 64 values minimum m and scale s = (maximum - m) / 15, both rounded to T, and codes rint((x - m) / s) cut to
// 0..15.  A group that holds infinities or NaN, spans more than a float, or has a minimum or scale beyond T is NaN as a whole
// (an infinite minimum with a finite scale would stand for 64 infinities, and a key of them can drop out of a softmax unseen).
template <class T, int D>
__device__ __forceinline__ void store_row4(char* codes, char* params, const LanePart& at, int l, bool live, const f2 (&v)[8]) {
    constexpr int LANES = D / 16;
    float low[2], high[2];
    ends_of(v, low[0], high[0]);
    ends_of(v + 4, low[1], high[1]);
    const int g0 = D > 64 ? at.c0 >> 3 : 0, g1 = D > 64 ? at.c1 >> 3 : 0;      // the pieces' groups
    // each half of the lanes ends with one group's ends (of two), or all with the one's
    const int mine = D > 64 ? l >> 2 : 0;
    float lo = fminf(g0 == mine ? low[0] : INFINITY, g1 == mine ? low[1] : INFINITY);
    float hi = max3(g0 == mine ? high[0] : -INFINITY, g1 == mine ? high[1] : -INFINITY, -INFINITY);
    if (D > 64) {
        const int other = mine ^ 1;
        const float lo2 = fminf(g0 == other ? low[0] : INFINITY, g1 == other ? low[1] : INFINITY);
        const float hi2 = max3(g0 == other ? high[0] : -INFINITY, g1 == other ? high[1] : -INFINITY, -INFINITY);
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo2, 4));
        const float x = __shfl_xor_sync(0xffffffffu, hi2, 4);
        hi = max3(hi, x, x);
    }
#pragma unroll
    for (int o = 2; o; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        const float x = __shfl_xor_sync(0xffffffffu, hi, o);
        hi = max3(hi, x, x);
    }
    const float scale = __fmul_rn(hi - lo, 1.0f / 15.0f);  // NaN, or infinite, with what is not finite
    constexpr float END = Pair<T>::bf16 ? 0x1.ffp127f : 65520.0f;      // what rounds to an infinity of T
    const bool fine = scale < END && fabsf(lo) < END;
    const uint32_t pair = Pair<T>::pack(fine ? scale : NAN, fine ? lo : NAN);
    const uint32_t p0 = D > 64 ? __shfl_sync(0xffffffffu, pair, 4 * g0, LANES) : pair;
    const uint32_t p1 = D > 64 ? __shfl_sync(0xffffffffu, pair, 4 * g1, LANES) : pair;
    const float2 s0 = Pair<T>::unpack(p0), s1 = Pair<T>::unpack(p1);
    const uint32_t w0 = codes_of(v, s0.x, s0.y), w1 = codes_of(v + 4, s1.x, s1.y);
    if (!live) return;
    reinterpret_cast<uint32_t*>(codes)[at.c0] = w0;
    reinterpret_cast<uint32_t*>(codes)[at.c1] = w1;
    if ((l & 3) == 0) reinterpret_cast<uint32_t*>(params)[mine] = pair;
}

// ---------------------------------------------------------------------------
// Forward, and the cache writes
// ---------------------------------------------------------------------------
enum Sink : int { kSinkRows, kSinkCache16, kSinkCache4 };

template <class T, int D, int SINK, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kCtasAnSm) gsr_rope_kernel(const __grid_constant__ RopeAppendParams a,
                                                                       const __grid_constant__ RopePlan plan) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES, N = SINK == kSinkRows ? 1 : 2;
    constexpr int STAGES = N == 1 ? 4 : 3;
    __shared__ uint4 s_ring[kWarps][STAGES][2 * N][32];
    const RopeParams& p = a.f;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, row = lane / LANES;
    const LanePart at_qk = lane_part<LANES, INTERLEAVED>(l, p.table ? p.R : 0), at_v = lane_part<LANES, false>(l, 0);
    auto rows = [&](int part, int n, LanePart& at) {
        at = n ? at_v : at_qk;
        if (n) return part ? a.V : Strided{nullptr, 0, 0, 0};
        return pick(part == 0, p.Q, p.K);
    };
    auto heads = [&](int part) { return part == 0 ? p.Hq : p.Hkv; };
    Walk now(plan, blockIdx.x * kWarps + warp, gridDim.x * kWarps);
    Ring<N, STAGES> ring(s_ring[warp], lane, now);
    auto load = [&] { ring.template load<ROWS>(plan, row, rows, heads); };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) load();

    TokenAngles turned;
    f2 w[8];
    // norm and rotation of a row of Q or K
    auto normed = [&](const uint4& lo, const uint4& hi, const void* weight, f2 (&v)[8]) {
        unpack_part<T>(lo, hi, v);
        if (weight) {
            f2 sum = mul2(v[0], v[0]);
#pragma unroll
            for (int k = 1; k < 8; ++k) sum = fma2(v[k], v[k], sum);
            const f2 r = both(rsqrtf(row_sum<LANES>(sum_of(sum)) * (1.0f / D) + p.eps));
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = mul2(mul2(v[k], r), w[k]);
        }
        if (turned.known) rotate<SINK == kSinkCache4, INTERLEAVED>(v, turned.angles, at_qk);
        else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = both(turned.pos < 0 ? 0.0f : NAN);
        }
    };
    auto store = [&](char* to, const LanePart& at, const f2 (&v)[8]) {
        reinterpret_cast<uint4*>(to)[at.c0] = pack_piece<T>(v);
        reinterpret_cast<uint4*>(to)[at.c1] = pack_piece<T>(v + 4);
    };
    while (now.left > 0) {
        now.open(plan, ROWS);
        const bool to_cache = SINK != kSinkRows && now.part > 0;
        const int slot = to_cache ? __ldg(a.slots + now.token) : 0;
        turned.template move<false, LANES, INTERLEAVED>(p, now.token, now.s, at_qk, l);
        const void* weight = now.part == 0 ? p.q_weight : p.k_weight;
        if (weight) load_weight<T>(weight, at_qk, w);
        const int h = now.h0 + row;
        int live = heads(now.part) - h;
        if (!to_cache) {
            const Strided t = pick(now.part == 0, p.Qo, p.Ko);
            char* to = static_cast<char*>(t.data) + 2 * (now.b * t.batch + now.s * t.row + h * t.head);
#pragma unroll 1
            for (; now.run > 0; --now.run) {
                load();
                ring.wait();
                uint4 lo, hi;
                ring.read(0, lo, hi);
                ring.advance();
                f2 v[8];
                normed(lo, hi, weight, v);
                if (live > 0) store(to, at_qk, v);
                to += 2 * ROWS * t.head;
                live -= ROWS;
            }
            continue;
        }
        const bool skip = slot < 0 || slot >= (long long)a.num_pages * a.page || (p.table && turned.pos < 0);      // padding
        const int page = plan.by_page(skip ? 0 : slot), r = (skip ? 0 : slot) - page * a.page;
        // where the lane's rows of K and V go
        char *to[2], *params[2] = {nullptr, nullptr};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            if (SINK == kSinkCache16) {
                const Strided& t = n ? a.Vc : a.Kc;
                to[n] = static_cast<char*>(t.data) + 2 * (page * t.batch + r * t.row + h * t.head);
            } else {
                const Cache4& t = n ? a.V4 : a.K4;
                to[n] = t.codes.data + page * t.codes.page + r * t.codes.row + h * t.codes.head;
                params[n] = t.params.data + page * t.params.page + r * t.params.row + h * t.params.head;
            }
        }
#pragma unroll 1
        for (; now.run > 0; --now.run) {
            load();
            ring.wait();
            uint4 lo, hi, v_lo, v_hi;
            ring.read(0, lo, hi);
            ring.read(N - 1, v_lo, v_hi);
            ring.advance();
            if (!skip) {
                f2 v[8];
                normed(lo, hi, weight, v);
                if (SINK == kSinkCache16) {
                    if (live > 0) {
                        store(to[0], at_qk, v);
                        reinterpret_cast<uint4*>(to[1])[at_v.c0] = v_lo;
                        reinterpret_cast<uint4*>(to[1])[at_v.c1] = v_hi;
                    }
                } else {
                    store_row4<T, D>(to[0], params[0], at_qk, l, live > 0, v);
                    unpack_part<T>(v_lo, v_hi, v);
                    store_row4<T, D>(to[1], params[1], at_v, l, live > 0, v);
                }
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                to[n] += SINK == kSinkCache16 ? 2 * ROWS * (n ? a.Vc : a.Kc).head : ROWS * (n ? a.V4 : a.K4).codes.head;
                params[n] += ROWS * (n ? a.V4 : a.K4).params.head;
            }
            live -= ROWS;
        }
    }
}

// CTAs of `units` steps: what fits on the SMs at once, or a step a warp.
int rope_ctas(long long units, int sms) {
    const long long ctas = (units + kWarps - 1) / kWarps;
    return (int)(ctas < (long long)kCtasAnSm * sms ? ctas : (long long)kCtasAnSm * sms);
}

RopePlan rope_plan(const RopeParams& p, int q_heads, int k_heads, int page) {
    const int rows = 512 / p.D;
    RopePlan plan{Divider(1), Divider((uint32_t)p.S), Divider((uint32_t)(page > 0 ? page : 1)), (q_heads + rows - 1) / rows,
                  (k_heads + rows - 1) / rows, 0};
    const int steps = plan.q_steps + plan.k_steps;
    if (steps > 0) plan.by_token = Divider((uint32_t)steps);
    plan.units = (int)((long long)p.B * p.S * steps);
    return plan;
}

template <class T, int D, int SINK>
cudaError_t launch_rope(const RopeAppendParams& a, int sms, cudaStream_t stream) {
    const RopeParams& p = a.f;
    const RopePlan plan = rope_plan(p, p.Hq, p.Hkv, a.page);
    const unsigned ctas = (unsigned)rope_ctas(plan.units, sms);
    if (p.table && p.interleaved) gsr_rope_kernel<T, D, SINK, true><<<ctas, kThreads, 0, stream>>>(a, plan);
    else gsr_rope_kernel<T, D, SINK, false><<<ctas, kThreads, 0, stream>>>(a, plan);
    return cudaGetLastError();
}
template <int SINK>
cudaError_t launch_rope_type(const RopeAppendParams& a, bool bf16, int sms, cudaStream_t stream) {
    if (a.f.D == 64)
        return bf16 ? launch_rope<__nv_bfloat16, 64, SINK>(a, sms, stream) : launch_rope<__half, 64, SINK>(a, sms, stream);
    return bf16 ? launch_rope<__nv_bfloat16, 128, SINK>(a, sms, stream) : launch_rope<__half, 128, SINK>(a, sms, stream);
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------
// With dy the incoming gradient turned back, n = x r, dn = dy w:
//   dw = sum over rows of dy n,   dx = r (dn - n mean(dn n)) = r dn - x r^3 sum(dn x) / D.
// r is computed again from x, which has to be read anyway, so the forward pass stores nothing.  A CTA sums dw
// over its rows in registers (fp32, a lane's 16 columns), then over its warps; a second launch adds the CTAs'
// sums in their order, so that results repeat.
constexpr int kBwdStages = 3;

// One step after another of a warp's share.
struct Cursor {
    int left, token, b, s, block;       // steps left; the token, its batch row and place; the step in the token
    __device__ __forceinline__ Cursor(const RopePlan& plan, int w, int warps) {
        const int each = (plan.units + warps - 1) / warps, first = (int)min((long long)w * each, (long long)plan.units);
        left = min(each, plan.units - first);
        token = plan.by_token(first);
        block = first - token * (int)plan.by_token.d;
        b = plan.by_seq(token);
        s = token - b * (int)plan.by_seq.d;
    }
    __device__ __forceinline__ void step(const RopePlan& plan) {
        --left;
        if (++block < plan.q_steps) return;
        block = 0;
        ++token;
        if (++s == (int)plan.by_seq.d) {
            s = 0;
            ++b;
        }
    }
};

// The rows of Q, or those of K.
template <class T, int D, bool INTERLEAVED, bool K_PART>
__device__ __forceinline__ void rope_bwd_part(const RopeBwdParams& a, const RopePlan& plan, uint4 (&s_ring)[kWarps][kBwdStages][4][32],
                                              const LanePart& at) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;
    float* const sums = reinterpret_cast<float*>(s_ring);  // of the warps, after the rows: D each
    const RopeParams& p = a.f;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES, row = lane / LANES;
    const Strided &G = K_PART ? p.Ko : p.Qo, &X = K_PART ? p.K : p.Q, &dX = K_PART ? a.dK : a.dQ;
    const void* weight = K_PART ? p.k_weight : p.q_weight;
    const int heads = K_PART ? p.Hkv : p.Hq;
    f2 dw[8], w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[k] = 0ull;
    if (weight) load_weight<T>(weight, at, w);
    Cursor ahead(plan, blockIdx.x * kWarps + warp, gridDim.x * kWarps), now = ahead;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(&s_ring[warp][0][0][lane]);
    uint32_t to = base, from = base;
    auto after = [&](uint32_t stage) { return stage == base + (kBwdStages - 1) * 2048 ? base : stage + 2048; };
    // addresses are computed for each step: kept from step to step they would spill
    auto load = [&] {
        if (ahead.left > 0) {
            const int h = ahead.block * ROWS + row;
            if (h < heads) {
                const uint4* g = reinterpret_cast<const uint4*>(static_cast<const T*>(G.data) + ahead.b * G.batch + ahead.s * G.row + h * G.head);
                copy_piece(to, g + at.c0);
                copy_piece(to + 512, g + at.c1);
                if (weight) {
                    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(X.data) + ahead.b * X.batch + ahead.s * X.row + h * X.head);
                    copy_piece(to + 1024, x + at.c0);
                    copy_piece(to + 1536, x + at.c1);
                }
            }
            ahead.step(plan);
            to = after(to);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kBwdStages - 1; ++i) load();
    TokenAngles turned;
#pragma unroll 1
    for (; now.left > 0; now.step(plan)) {
        load();
        turned.template move<true, LANES, INTERLEAVED>(p, now.token, now.s, at, l);
        const int h = now.block * ROWS + row;
        const bool counts = h < heads && (!p.table || turned.pos >= 0);       // padding adds nothing, whatever it holds
        asm volatile("cp.async.wait_group %0;" ::"n"(kBwdStages - 1) : "memory");
        f2 dy[8];
        unpack_part<T>(ring_piece(from), ring_piece(from + 512), dy);
        if (turned.known) rotate<false, INTERLEAVED>(dy, turned.angles, at);
        else {
#pragma unroll
            for (int k = 0; k < 8; ++k) dy[k] = both(NAN);
        }
        if (weight) {
            f2 v[8], square = 0ull, dot = 0ull;
            unpack_part<T>(ring_piece(from + 1024), ring_piece(from + 1536), v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                square = fma2(v[k], v[k], square);
                dot = fma2(mul2(dy[k], w[k]), v[k], dot);
            }
            const float r = rsqrtf(row_sum<LANES>(sum_of(square)) * (1.0f / D) + p.eps);
            const float back = row_sum<LANES>(sum_of(dot)) * (1.0f / D) * r * r * r;
            const f2 rr = both(r), minus = both(-back);
            if (counts) {
#pragma unroll
                for (int k = 0; k < 8; ++k) dw[k] = fma2(mul2(dy[k], v[k]), rr, dw[k]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) dy[k] = fma2(v[k], minus, mul2(mul2(dy[k], w[k]), rr));
        }
        from = after(from);
        if (h < heads) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(dX.data) + now.b * dX.batch + now.s * dX.row + h * dX.head);
            const uint4 none = make_uint4(0u, 0u, 0u, 0u);
            out[at.c0] = counts ? pack_piece<T>(dy) : none;
            out[at.c1] = counts ? pack_piece<T>(dy + 4) : none;
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // What the call has parts for: a weight whose rows have no heads may come without its gradient.
    if (!(K_PART ? a.dk_weight : a.dq_weight)) return;
    float sum[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 x = parts_of(dw[k]);
        sum[2 * k] = x.x;
        sum[2 * k + 1] = x.y;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
    __syncthreads();
    if (lane < LANES) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sums[warp * D + 8 * at.c0 + k] = sum[k];
            sums[warp * D + 8 * at.c1 + k] = sum[8 + k];
        }
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) t += sums[k * D + threadIdx.x];
        a.parts[((long long)K_PART * a.ctas + blockIdx.x) * D + threadIdx.x] = t;
    }
    __syncthreads();
}

template <class T, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kCtasAnSm) gsr_rope_bwd_kernel(const __grid_constant__ RopeBwdParams a,
                                                                           const __grid_constant__ RopePlan q_plan,
                                                                           const __grid_constant__ RopePlan k_plan) {
    __shared__ uint4 s_ring[kWarps][kBwdStages][4][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const LanePart at = lane_part<D / 16, INTERLEAVED>(threadIdx.x % (D / 16), a.f.table ? a.f.R : 0);
    rope_bwd_part<T, D, INTERLEAVED, false>(a, q_plan, s_ring, at);
    rope_bwd_part<T, D, INTERLEAVED, true>(a, k_plan, s_ring, at);
}

// dw = sum of the CTAs' parts, a CTA for 32 columns: 32 lanes of rows, each in ascending order.
__global__ void __launch_bounds__(1024) gsr_rope_weights_kernel(const float* parts, int ctas, int D, float* dq_weight, float* dk_weight) {
    __shared__ float sums[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");     // launched while the rows' CTAs run
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    float* to = blockIdx.y ? dk_weight : dq_weight;
    if (!to) return;
    float t = 0.0f;
#pragma unroll 8
    for (int i = y; i < ctas; i += 32) t += parts[((long long)blockIdx.y * ctas + i) * D + col];
    sums[y][threadIdx.x & 31] = t;
    __syncthreads();
    if (y == 0) {
        t = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += sums[i][threadIdx.x];
        to[col] = t;
    }
}

template <class T, int D>
cudaError_t launch_bwd(const RopeBwdParams& a, cudaStream_t stream) {
    const RopeParams& p = a.f;
    cudaError_t e = cudaSuccess;
    if (a.ctas > 0) {
        const RopePlan q_plan = rope_plan(p, p.Hq, 0, 0), k_plan = rope_plan(p, p.Hkv, 0, 0);
        if (p.table && p.interleaved) gsr_rope_bwd_kernel<T, D, true><<<(unsigned)a.ctas, kThreads, 0, stream>>>(a, q_plan, k_plan);
        else gsr_rope_bwd_kernel<T, D, false><<<(unsigned)a.ctas, kThreads, 0, stream>>>(a, q_plan, k_plan);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.dq_weight || a.dk_weight) {
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute early;
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(D / 32, 2);
        cfg.blockDim = dim3(1024);
        cfg.stream = stream;
        cfg.attrs = &early;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, gsr_rope_weights_kernel, static_cast<const float*>(a.parts), a.ctas, D, a.dq_weight, a.dk_weight);
    }
    return e;
}

// ---------------------------------------------------------------------------
// Rows of a cache of 4 bits, read back
// ---------------------------------------------------------------------------
// 24576 tokens of 8 x 128 in 24 us: 129 MB, four fifths of a copy's rate.  A lane takes 16 values: 8 bytes of codes become
// 32 bytes.  s x code is exact in fp32, so a value is rounded once there and once to T.
template <class T, int D>
__global__ void __launch_bounds__(kThreads) gsr_read4_kernel(const __grid_constant__ Read4Params p, const Divider by_head,
                                                             const Divider by_page, long long rows) {
    constexpr int LANES = D / 16, PER = kThreads / LANES;
    const long long id = (long long)blockIdx.x * PER + threadIdx.x / LANES;      // a token's heads of K, then of V
    const int l = threadIdx.x % LANES;
    if (id >= rows) return;
    const bool is_v = id >= rows / 2;
    const int r = (int)(is_v ? id - rows / 2 : id), n = by_head(r), h = r - n * p.H;
    const int slot = __ldg(p.slots + n);
    if (slot < 0 || slot >= (long long)p.num_pages * p.page) return;
    const long long page = by_page(slot);
    const int row = slot - (int)page * p.page;
    const Cache4& cache = is_v ? p.V4 : p.K4;
    const Strided& to = is_v ? p.V : p.K;
    const uint2 codes = __ldg(reinterpret_cast<const uint2*>(cache.codes.data + page * cache.codes.page +
                                                             (long long)row * cache.codes.row + h * cache.codes.head) + l);
    const float2 sm = Pair<T>::unpack(__ldg(reinterpret_cast<const uint32_t*>(cache.params.data + page * cache.params.page +
                                                                             (long long)row * cache.params.row +
                                                                             h * cache.params.head) + l / 4));
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = fmaf(sm.x, (float)((i < 8 ? codes.x : codes.y) >> (4 * (i & 7)) & 15u), sm.y);
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(to.data) + n * to.row + h * to.head) + 2 * l;
    out[0] = pack8<T>(v);
    out[1] = pack8<T>(v + 8);
}

template <class T, int D>
cudaError_t launch_read(const Read4Params& p, cudaStream_t stream) {
    const long long rows = 2ll * p.N * p.H;
    constexpr int PER = kThreads / (D / 16);
    gsr_read4_kernel<T, D><<<(unsigned)((rows + PER - 1) / PER), kThreads, 0, stream>>>(p, Divider((uint32_t)p.H),
                                                                                        Divider((uint32_t)p.page), rows);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_fwd(const RopeParams& p, bool bf16, int sms, cudaStream_t stream) {
    RopeAppendParams a{};
    a.f = p;
    return launch_rope_type<kSinkRows>(a, bf16, sms, stream);
}

cudaError_t launch_rope_append(const RopeAppendParams& p, bool bf16, bool four_bits, int sms, cudaStream_t stream) {
    return four_bits ? launch_rope_type<kSinkCache4>(p, bf16, sms, stream) : launch_rope_type<kSinkCache16>(p, bf16, sms, stream);
}

int rope_bwd_ctas(long long batch, long long heads_q, long long heads_kv, long long seq, int D, int sms) {
    const int rows = 512 / D;
    return rope_ctas(batch * seq * (((heads_q > heads_kv ? heads_q : heads_kv) + rows - 1) / rows), sms);
}

cudaError_t launch_rope_bwd(const RopeBwdParams& p, bool bf16, cudaStream_t stream) {
    if (p.f.D == 64) return bf16 ? launch_bwd<__nv_bfloat16, 64>(p, stream) : launch_bwd<__half, 64>(p, stream);
    return bf16 ? launch_bwd<__nv_bfloat16, 128>(p, stream) : launch_bwd<__half, 128>(p, stream);
}

cudaError_t launch_read4(const Read4Params& p, bool bf16, cudaStream_t stream) {
    if (p.D == 64) return bf16 ? launch_read<__nv_bfloat16, 64>(p, stream) : launch_read<__half, 64>(p, stream);
    return bf16 ? launch_read<__nv_bfloat16, 128>(p, stream) : launch_read<__half, 128>(p, stream);
}

}  // namespace gsr
