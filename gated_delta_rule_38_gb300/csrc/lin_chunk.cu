// Linear attention with one decay lambda = exp(decay) a head, in chunks of 128 tokens on tcgen05:
//
//   S_t = lambda S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
//   a chunk of L tokens r, s from the state S before it:
//     P_rs = scale lambda^(r-s) q_r . k_s  (s <= r);   o = P V + diag(scale lambda^(r+1)) Q S
//     S <- lambda^L S + (diag(lambda^(L-1-s)) K)^T V
//
// The gradients are walks of the same form: dq = scale x the walk (do, v, k) from the transposed states, and backwards in
// time, where position r sees s >= r, dk = the walk (v, do, scale q) and dv = the walk (k, scale q, do) from the
// gradient of the final state, which has decayed by lambda^(L-1-r) at row r and by lambda^L at the chunk's start; the
// keys then enter the state with lambda^(s+1).  So one kernel runs the forward and, three walks side by side, the
// backward.
//
// One CTA walks one segment of a sequence for one head; all tiles are 128 wide (narrower heads load zeros).
//   warps 0..7    the state: lanes 32 (w mod 4) .., 64 of the 128 columns; fp32 in registers, with a copy rounded to 16 bits
//                 in shared memory as the operand of Q S; and the output rows
//   warps 8..11   lanes 32 (w mod 4) ..
//   all twelve    P from Q K^T (tensor memory to tensor memory, where it is the left operand of P V), in blocks of 32 x 32:
//                 warps 8..11 those on the diagonal and next to it, the others those beyond; then the decayed keys
//   warp 12       tile loads (TMA) into a ring of five 32 KB tiles
//   warp 13       the MMAs:  Q S, P V, the state's update, Q K^T of the next chunk
// The chain of a chunk: the update, the state's copy and the next Q S on one side, the next Q K^T and P on the other, then
// P V, and the next update; output rows and keys are made beside it.
// Fourteen warps leave a thread 128 registers; with eighteen and 96 the state's threads spilled, and what they spilled went
// to L2.  Loops that can stay loops do: unrolled, a chunk's code no longer fitted the instruction caches next to the
// schedulers.  (1 x 2048 tokens, 152 heads, one walk a CTA, 318 MB: 156 us with spills, 72 with sixteen warps through all
// steps together, 60 so, which is 5.3 TB/s, or 3.8 us a chunk; the matrix instructions take half of them.)
// The states inside are without their scale's power of two (of the gradients' walks), which the keys then need not carry.
// P and the state's copy are rounded to 16 bits, as operands of the tensor core: with the output's own rounding that makes
// outputs 1.4 times as far from 64 bits as one rounding would (bf16 2.3e-3, fp16 2.9e-4).  A second number for each would take
// two more products a chunk, and a 32 KB tile that shared memory does not have.
// A decayed key is a sum of 16-bit numbers, the rounded one and what that leaves, each with a product of its own, the
// smallest first: the accumulator loses at each addition by what it holds.  Two of fp16 make 22 bits and states 2e-7 off
// (of one number: 1e-3); the second is held times 2^11, or below a key of 0.1 it would be a subnormal number, and its
// products' sum is scaled back when the first number's are added (keys of 1e-3: states 2e-5 off without).  Two of bf16 make
// 17 bits and 2.5e-6, which outputs of 8 bits do not show; states that are handed on get a third where the chunk weighs over
// an eighth in them (3e-7).  Its place is the state's copy's, free between Q S and the next copy, and warps 8..11 make all the
// keys of such a chunk: the state's warps have no registers for it.  (2 x 4096 tokens, 32 heads of memories of 100 tokens: 88
// us with the final states, 79 without; where nothing decays, so that every chunk has three, 110.)  The products' loop stays
// a loop: with its bodies side by side the training step of 2 x 4096 tokens took 296 us, 287 so.
// The accumulators of one chunk's state update start from zero and are added to the state in fp32 registers, rounded to
// nearest: in the tensor core's own accumulator the additions of a long walk would lose in one direction.
// lambda^128 is kept as two fp32 numbers, so that a memory of any length is not off by what rounding it once would add up to.
//
// Segments.  Where sequences x heads leave SMs idle the token axis is cut; a first launch (STATES: no q, P or output rows, up to
// two chunks on their way) leaves every window's own end state, and a segment begins with the decayed sum of the windows
// before it, in a fixed order.  (1 x 65536 tokens, 16 heads: 99 us for the states and 215 for the walk, 4.8 TB/s in the first
// launch, which reads 8/9 of k and v.)
#include "common.cuh"
#include "f32x2.cuh"
#include "lin.h"
#include "seqwalk.cuh"
#include "umma.cuh"

namespace gdr {
namespace lin {
namespace {

constexpr int NS = 8, NK = 4, NT = 32 * (NS + NK + 2);  // warps of the state and of the keys; threads
constexpr int CW = LD / (NS / 4);                       // columns of a state warp
constexpr uint32_t TILE = 32768, BLK = 16384;     // a tile: two blocks of 64 columns, 128 rows each
constexpr int RING = 5;
constexpr uint32_t S_LO = RING * TILE;            // the keys' remainders
constexpr uint32_t S_ST = S_LO + TILE;            // the state's copy (state pass: the remainders of odd chunks); third numbers
constexpr uint32_t S_BAR = S_ST + TILE;
constexpr uint32_t B_FULL = S_BAR, B_EMPTY = S_BAR + 8 * RING, B_QK = B_EMPTY + 8 * RING, B_S = B_QK + 8, B_P = B_S + 8,
                   B_PV = B_P + 8, B_K = B_PV + 8, B_DS = B_K + 16, B_DONE = B_DS + 16, B_QS = B_DONE + 8, B_MAX = B_QS + 8,
                   S_SLOT = B_MAX + 16, S_FLAG = S_SLOT + 4;
constexpr uint32_t S_FROM = S_FLAG + 4;           // the first chunk whose decayed keys are three numbers
constexpr uint32_t S_LAM = S_FLAG + 8;            // lambda^128 as two fp32 numbers
// decays of up to 31 tokens: COL[c] = lambda^(31-c) (rev: lambda^c); DIAG[31 + row - key] = s_kv s_out lambda^|row - key| where
// the row sees the key, else 0
constexpr uint32_t S_COL = (S_LAM + 8 + 15) / 16 * 16, S_DIAG = S_COL + 128;
// fp16: the largest magnitude in each state warp's part of the state, by parity of the chunk; four warps of the same columns
// side by side
constexpr uint32_t S_MAX = S_DIAG + 256;
constexpr uint32_t S_BYTES = S_MAX + 8 * NS + 1024;
static_assert(S_BYTES <= kSmemMost, "shared memory");
// tensor memory columns: Q K^T and, in its place, P (each 32 columns in the lower half of their own); Q S; P V; the update
constexpr uint32_t T_QK = 0, T_QS = 128, T_PV = 256, T_DS = 384;

template <int N> struct Int { static constexpr int value = N; };
template <typename T> struct IsBf16 { static constexpr bool value = false; };
template <> struct IsBf16<__nv_bfloat16> { static constexpr bool value = true; };

// ---------------------------------------------------------------- waits

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t lds32_now(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float lds_f(uint32_t addr) { return __uint_as_float(lds32(addr)); }
constexpr unsigned long long kWaitNs = 2000000000ull;
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;\n" : "=l"(t));
    return t;
}
__device__ __forceinline__ bool try_phase(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
// Waits for a barrier's phase; gives up when another role raised the block's flag, or after two seconds (then it raises it).
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, uint32_t flag, unsigned *err) {
    if (try_phase(bar, parity)) return true;
    const unsigned long long from = now_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i)
            if (try_phase(bar, parity)) return true;
        if (lds32_now(flag)) return false;
        if (now_ns() - from > kWaitNs) break;
    }
    raise_error(err, GDR_ERR_TIMEOUT);
    sts32(flag, 1);
    return false;
}
// Two or three at once: their tests overlap.
__device__ __forceinline__ bool wait_phases(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2, uint32_t flag, unsigned *err) {
    const bool r0 = try_phase(b0, p0), r1 = try_phase(b1, p1), r2 = try_phase(b2, p2);
    return (r0 || wait_phase(b0, p0, flag, err)) && (r1 || wait_phase(b1, p1, flag, err)) && (r2 || wait_phase(b2, p2, flag, err));
}
// Every lane polls and the warp agrees on the outcome.
__device__ __forceinline__ bool wwait(uint32_t bar, uint32_t parity, uint32_t flag, unsigned *err) {
    return __all_sync(0xffffffffu, wait_phase(bar, parity, flag, err));
}

// ---------------------------------------------------------------- tensor memory

// 32 lanes x 32 columns; the wait names the registers, so that nothing that uses them moves above it.
__device__ __forceinline__ void tld32(uint32_t a, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
}
__device__ __forceinline__ void twait16(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void twait32(uint32_t *r) {
    twait16(r);
    twait16(r + 16);
}
__device__ __forceinline__ void tld16(uint32_t a, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
}
__device__ __forceinline__ void tst8(uint32_t a, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tst16(uint32_t a, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tst_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// D (+)= A B, issued by the lane that has `on`; the whole warp computes the operands, which so stay uniform.  (In a branch
// of one lane every MMA took 100 cycles to issue, half as long again as it runs.)
__device__ __forceinline__ void mma_ss(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool accumulate) {
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"((uint32_t)accumulate), "r"(on));
}
// D = A B + D / 2^11.
constexpr float kLoScale = 2048.f;
__device__ __forceinline__ void mma_ss_down(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.eq.b32 p, %4, %4;\nsetp.ne.b32 q, %4, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p, 11;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(on));
}
// ... with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool accumulate) {
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"((uint32_t)accumulate), "r"(on));
}
__device__ __forceinline__ void commit_on(uint32_t on, uint32_t bar) {
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(on));
}
// A descriptor's words: the upper one is the same for every step of an operand, the lower one moves on by 16 bytes each.
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) {
    const uint32_t lo = (uint32_t)d + (bytes >> 4), hi = (uint32_t)(d >> 32);
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
// 32 bytes of one row, from a 32-byte boundary.
__device__ __forceinline__ void store32(void *p, f2 a, f2 b, f2 c, f2 d) {
    asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};\n" ::"l"(p), "l"(a), "l"(b), "l"(c), "l"(d) : "memory");
}
__device__ __forceinline__ f2 f2_of(uint32_t lo, uint32_t hi) {
    return pack2(__uint_as_float(lo), __uint_as_float(hi));
}

// ---------------------------------------------------------------- segments

struct Seg {
    int n;           // sequence, -1: none
    int t0, t1;      // its tokens, of all rows
    int seq0, seq1;  // the sequence's
};
// Cuts of one length over the sequences.
struct Cuts {
    const LinArgs &a;
    int len;
    __device__ __forceinline__ Cuts(const LinArgs &a_, int len_) : a(a_), len(len_) {}
    __device__ __forceinline__ int per() const { return a.T > 0 ? (int)((a.T + (long long)len - 1) / len) : 1; }
    __device__ __forceinline__ int cu(int n) const { return min(max(a.cu[n], 0), a.T); }
    // The segment at a place.  Packed: sequence starts and multiples of len in one sorted order (of equal ones the
    // starts first); the piece from one to the next.  In range whatever cu holds.
    __device__ Seg at(int slot) const {
        Seg s;
        if (!a.cu) {
            const int w = per();
            s.n = slot / w;
            const int i = slot - s.n * w;
            s.seq0 = s.n * a.T;
            s.seq1 = s.seq0 + a.T;
            s.t0 = s.seq0 + (int)min((long long)i * len, (long long)a.T);
            s.t1 = s.seq0 + (int)min((i + 1ll) * len, (long long)a.T);
            return s;
        }
        // the first `slot` of the sorted order hold p starts: the smallest p with start p behind multiple slot - 1 - p
        int lo = max(0, slot - (a.T > 0 ? per() : 0)), hi = min(slot, a.N);
        while (lo < hi) {
            const int p = (lo + hi) >> 1;
            if ((long long)cu(p) > (long long)(slot - 1 - p) * len) hi = p;
            else lo = p + 1;
        }
        int p = lo, q = slot - lo;
        const int W = a.T > 0 ? per() : 0;
        const bool start = p < a.N && (q >= W || (long long)cu(p) <= (long long)q * len);
        s.t0 = start ? cu(p) : (int)min((long long)q * len, (long long)a.T);
        if (start) ++p; else ++q;
        s.n = p - 1;
        s.seq0 = s.seq1 = 0;
        s.t1 = s.t0;
        if (s.n < 0) return s;
        s.seq0 = cu(s.n);
        s.seq1 = max(cu(s.n + 1), s.seq0);
        s.t1 = min(s.seq1, q < W ? (int)min((long long)q * len, (long long)a.T) : a.T);
        if (s.t1 < s.t0 || s.t0 < s.seq0) s.t1 = s.t0;
        // (an empty piece belongs to its sequence only if that is empty: then it hands the state through)
        if (s.t1 == s.t0 && !(start && s.seq1 == s.seq0)) s.n = -1;
        return s;
    }
    // Within a sequence: the next cut behind t, the last one at or before it, and the place of the exchanged state of the piece
    // that begins at t.  Packed: the interval of the token axis that it lies in (its place in the order, less the starts before).
    // Of the pieces in one interval a segment only ever wants one, the one whose sequence goes on behind it (backwards: before
    // it).
    __device__ __forceinline__ int base(const Seg &s) const { return a.cu ? 0 : s.seq0; }
    __device__ __forceinline__ int next(const Seg &s, int t) const {
        const long long c = base(s) + ((long long)(t - base(s)) / len + 1) * len;
        return (int)min(c, (long long)s.seq1);
    }
    __device__ __forceinline__ int last(const Seg &s, int t) const { return base(s) + (t - base(s)) / len * len; }
    __device__ __forceinline__ long long place(const Seg &s, int t) const {
        return a.cu ? t / len : (long long)s.n * per() + (t - s.seq0) / len;
    }
};

// ---------------------------------------------------------------- the kernel

// MAY: keys of three numbers.
template <typename T, bool STATES, bool MAY>
__global__ void __launch_bounds__(NT, 1) lin_walk_kernel(const __grid_constant__ LinParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const LinArgs &a = p.a;
    const unsigned item = blockIdx.x;
    const int wi = (int)(item % (unsigned)a.nwalk);
    const unsigned rest = item / (unsigned)a.nwalk;
    const int j = (int)(rest % (unsigned)a.H), slot = (int)(rest / (unsigned)a.H);
    const Walk &w = p.w[wi];
    const bool rev = w.rev;
    const int kd = w.kd, vd = w.vd;
    if (blockIdx.x == 0 && a.cu) check_cu(a.cu, a.N, a.T, a.err);

    const Cuts cuts(a, STATES ? a.win_len : a.main_len);
    const Seg seg = cuts.at(slot);
    if (seg.n < 0) return;
    bool at_start = rev ? seg.t1 == seg.seq1 : seg.t0 == seg.seq0;  // the walk begins (ends) with this segment
    bool at_end = rev ? seg.t0 == seg.seq0 : seg.t1 == seg.seq1;
    if (STATES) {
        // a window's state is wanted where a segment begins behind it
        const Cuts mc(a, a.main_len);
        if (rev ? mc.last(seg, seg.t0) <= seg.seq0 : mc.next(seg, seg.t0) >= seg.seq1) return;
    }
    const int nc = (seg.t1 - seg.t0 + LC - 1) / LC;
    if (nc == 0 && !(w.end != nullptr)) return;
    const bool has_start = !STATES && (w.start != nullptr || !at_start);
    const bool want_end = STATES || (w.end != nullptr && at_end);
    const uint32_t flag = sb + S_FLAG;
    const float g = a.decay[j] < -120.f ? -120.f : a.decay[j];  // (e^-120 is 0 in fp32; 0 x -inf would be NaN)
    const float lg = g * LOG2E;

    // chunk c of the walk: its first token and length
    auto chunk = [&](int c, int &t, int &L) {
        t = seg.t0 + (rev ? nc - 1 - c : c) * LC;
        L = min(LC, seg.t1 - t);
    };
    constexpr int PER = STATES ? 2 : 3;  // tiles a chunk: (q,) k, v
    auto slot_of = [&](int c, int which) { return (PER * c + which) % RING; };
    auto phase_of = [&](int c, int which) { return (uint32_t)(((PER * c + which) / RING) & 1); };
    constexpr int KI = STATES ? 0 : 1, VI = KI + 1;
    const int kblk = kd > 64 ? 2 : 1, vblk = vd > 64 ? 2 : 1;
    // a chunk's tile into its place of the ring
    auto tile = [&](int c, int i) {
        int t, L;
        chunk(c, t, L);
        const CUtensorMap *m = i == VI ? &w.tv : i == KI ? &w.tk : &w.tq;
        const int h = j / (i == VI ? w.v_div : i == KI ? w.k_div : w.q_div), nb = i == VI ? vblk : kblk;
        if (lane == 0) {
            const uint32_t dst = sb + slot_of(c, i) * TILE, bar = sb + B_FULL + 8 * slot_of(c, i);
            tma::expect_tx(bar, nb * BLK);
#pragma unroll 1
            for (int b = 0; b < nb; ++b) tma::load3d(dst + b * BLK, m, 64 * b, h, t, bar);
        }
        __syncwarp();
    };
    // The loading warp prepares the barriers and begins with the first chunk while the others prepare the rest.
    if (warp == NS + NK) {
        if (lane == 0) {
            for (int i = 0; i < RING; ++i) {
                umma::mbar_init(sb + B_FULL + 8 * i, 1);
                umma::mbar_init(sb + B_EMPTY + 8 * i, 1);
            }
            umma::mbar_init(sb + B_QK, 2);
            umma::mbar_init(sb + B_PV, 1);
            umma::mbar_init(sb + B_P, NS + NK);
            umma::mbar_init(sb + B_S, NS);
            for (int i = 0; i < 2; ++i) {
                umma::mbar_init(sb + B_K + 8 * i, NS + NK);
                umma::mbar_init(sb + B_DS + 8 * i, 1);
            }
            umma::mbar_init(sb + B_DONE, 1);
            umma::mbar_init(sb + B_QS, 1);
            for (int i = 0; i < 2; ++i) umma::mbar_init(sb + B_MAX + 8 * i, 4);
            umma::fence_mbar_init();
            sts32(flag, 0);
        }
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < PER && nc > 0; ++i) tile(0, i);
    }
    if (tid == 32) {
        const double l = exp((double)g * LC);
        sts32(sb + S_LAM, __float_as_uint((float)l));
        sts32(sb + S_LAM + 4, __float_as_uint((float)(l - (double)(float)l)));
        int from = 0x7fffffff;
        if (w.end) {  // tokens after which an eighth is left, and those behind the segment's first one
            const float reach = lg < 0.f ? -3.f / lg : 2e9f, ahead = (float)(rev ? seg.t1 - seg.seq0 : seg.seq1 - seg.t0);
            if (!STATES) from = max((int)((ahead - reach) * (1.f / LC)), 0);
            else if (ahead - (float)(seg.t1 - seg.t0) < reach) from = 0;
        }
        sts32(sb + S_FROM, (uint32_t)from);
    }
    if (tid >= 64 && tid < 96) reinterpret_cast<float *>(smem + S_COL)[lane] = ex2((float)(rev ? lane : 31 - lane) * lg);
    if (tid >= 96 && tid < 160) {
        const int d = rev ? 31 - (tid - 96) : tid - 96 - 31;
        reinterpret_cast<float *>(smem + S_DIAG)[tid - 96] = d >= 0 ? w.s_kv * w.s_out * ex2((float)d * lg) : 0.f;
    }
    if (warp == NS + NK + 1) umma::alloc(sb + S_SLOT, 512);
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + S_SLOT);

    // Whether chunk c's decayed keys are three numbers (once so, then to the walk's end; the state pass: its whole window).
    auto three = [&](int c) { return MAY && c >= (int)lds32_now(sb + S_FROM); };
    // The state pass' hand-offs run up to two chunks ahead of one another, so each parity of chunks has its own barriers.
    auto bar_of = [&](uint32_t bar, int c) { return sb + bar + (STATES && (c & 1) ? 8u : 0u); };
    auto par_of = [&](int c) { return (uint32_t)((STATES ? c >> 1 : c) & 1); };
    const int ksteps = (kd + 15) / 16;
    const int NV = (vd + 15) / 16 * 16;

    // The keys' remainders of chunk c.
    auto lo_of = [&](int c) { return STATES && (c & 1) && !three(c) ? S_ST : S_LO; };
    // The decayed keys of chunk c, eights i0 .. i1 of the columns of row 32 (warp mod 4) + lane; the rounded ones in place of k.
    auto make_keys = [&](int c, int L, int i0, int i1, auto all) {
        const int row = (warp & 3) * 32 + lane;
        const uint32_t kt = sb + slot_of(c, KI) * TILE, lo = sb + lo_of(c);
        const bool in = row < L;
        const float f = in ? w.s_key * ex2((float)(rev ? row + 1 : L - 1 - row) * lg) : 0.f;  // (behind the end it could be infinite)
        auto place = [&](int i) { return (uint32_t)(i >> 3) * BLK + row * 128 + (((uint32_t)(i & 7) ^ (row & 7)) << 4); };
        // N eights at a time, as M numbers each
        auto convert = [&](int from, int to, auto n, auto terms) {
            constexpr int N = decltype(n)::value, M = decltype(terms)::value;
#pragma unroll 1
            for (int i = from; i < to; i += N) {
                uint4 u[N];
                uint32_t at[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    at[k] = (uint32_t)(i >> 3) * BLK + row * 128 + (((uint32_t)((i & 7) + k) ^ (row & 7)) << 4);
                    u[k] = umma::ld_shared_v4(kt + at[k]);
                    if (!in) u[k] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const uint32_t x[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
                    uint32_t h[4], l[4], m[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f2 v = mul2(widen2<T>(x[e]), both(f));
                        h[e] = narrow2<T>(v);
                        const f2 r = fma2(widen2<T>(h[e]), both(-1.f), v);
                        l[e] = narrow2<T>(IsBf16<T>::value ? r : mul2(r, both(kLoScale)));
                        if (M == 3) m[e] = narrow2<T>(fma2(widen2<T>(l[e]), both(-1.f), r));
                    }
                    umma::st_shared_v4(kt + at[k], h[0], h[1], h[2], h[3]);
                    umma::st_shared_v4(lo + at[k], l[0], l[1], l[2], l[3]);
                    if (M == 3) umma::st_shared_v4(sb + S_ST + at[k], m[0], m[1], m[2], m[3]);
                }
            }
        };
        if (decltype(all)::value && three(c)) convert(0, 8 * kblk, Int<4>(), Int<3>());
        else convert(i0, i1, Int<2>(), Int<2>());
        umma::fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_of(B_K, c));
    };

    // The state's copy is of the tokens' type.  In fp16 it is taken times a power of two that brings the largest of the 64 columns
    // that four warps share to between 2^14 and 2^15: the state itself may lie far outside that type's range.  The output rows
    // take the power back; it follows from the warps' maxima, so that no thread has to keep it.  A maximum is of finite numbers:
    // twice their bits and one more in the exponent, which for the others wraps to zero's or less.  (Capped where fp32's range
    // ends.  2 x 4096 tokens, 32 heads: 95 us; 87 without, and with states past 65504 infinite.  Maxima of pairs of the rounded
    // copy, of three numbers an instruction, or asked for only when the copy's product has begun: 95 to 98.)
    auto maxima = [&](int c) { return sb + S_MAX + (uint32_t)((c & 1) * NS + ((warp >> 2) & 1) * 4) * 4; };
    auto copy_shift = [&](int c) {
        const uint4 m = umma::ld_shared_v4(maxima(c));
        return min(127 + 1 + 14 - (int)(max(max(m.x, m.y), max(m.z, m.w)) >> 24), 100);
    };
    auto two_to = [](int e) { return __uint_as_float((uint32_t)(127 + e) << 23); };

    // The block of P `dist` blocks of 32 from the diagonal in this warp's rows, if there is one: lambda^|r-s| as a row's factor
    // (distance to the block's near edge) times a column's (from there), both at most 1.
    auto p_beyond = [&](int dist, int L) {
        const int q4 = warp & 3, blk = rev ? q4 + dist : q4 - dist;
        if (blk < 0 || blk > 3) return;
        const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16) + T_QK + 32 * blk;
        const f2 rf = both(w.s_kv * w.s_out * ex2((float)(32 * dist + (rev ? -lane : lane - 31)) * lg));
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            uint32_t x[16], o[8];
            float4 f[4];
            tld16(at + 16 * h, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = reinterpret_cast<const float4 *>(smem + S_COL)[4 * h + i];
            twait16(x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[2 * i] = narrow2<T>(mul2(mul2(f2_of(x[4 * i], x[4 * i + 1]), rf), pack2(f[i].x, f[i].y)));
                o[2 * i + 1] = narrow2<T>(mul2(mul2(f2_of(x[4 * i + 2], x[4 * i + 3]), rf), pack2(f[i].z, f[i].w)));
            }
            if (rev && L < LC) {  // (a short chunk's rows see no keys behind it)
                const int most = L - 32 * blk - 16 * h;
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = 2 * i + 1 < most ? o[i] : 2 * i < most ? o[i] & 0xffffu : 0u;
            }
            // (columns of this block that it has read: the lower 16 of its 32)
            tst8(at + 8 * h, o);
        }
    };

    // The output rows of chunk c, columns c0 .. c1 (multiples of 16) of row 32 (warp mod 4) + lane.  Rows of 16 columns are whole
    // 32-byte sectors where they begin on one.  (A lane has a row of its own.  A tile staged for a TMA store kept its place from
    // the loads, and the next chunk's v came late.)
    auto out_rows = [&](int c, int t, int L, int c0, int c1) {
        const int row = (warp & 3) * 32 + lane;
        const uint32_t quad = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const bool use_s = c > 0 || has_start;
        umma::fence_after();
        float rf = use_s ? w.s_out * w.s_state * ex2((float)(rev ? L - 1 - row : row + 1) * lg) : 0.f;
        if (!IsBf16<T>::value) rf *= two_to(-copy_shift(c));
        const long long at = (((long long)t + row) * a.H + j) * vd;
        const bool wide = row < L && vd % 16 == 0 && reinterpret_cast<uintptr_t>(w.out) % 32 == 0;
#pragma unroll 1
        for (int col = c0; col < c1 && col < vd; col += 16) {
            uint32_t x[16], y[16];
            tld16(quad + T_PV + col, x);
            if (use_s) tld16(quad + T_QS + col, y);
            twait16(x);
            f2 v[8];  // (P has both factors; Q S gets them, and the decay, here)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = f2_of(x[2 * e], x[2 * e + 1]);
            if (use_s) {
                twait16(y);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = fma2(f2_of(y[2 * e], y[2 * e + 1]), both(rf), v[e]);
            }
            if (w.out_f32) {
                float *o = static_cast<float *>(w.out) + at + col;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (row < L && col + 8 * e < vd) store32(o + 8 * e, v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            } else {
                T *o = static_cast<T *>(w.out) + at + col;
                uint32_t u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = narrow2<T>(v[e]);
                if (wide) {
                    store32(o, (f2)u[1] << 32 | u[0], (f2)u[3] << 32 | u[2], (f2)u[5] << 32 | u[4], (f2)u[7] << 32 | u[6]);
                } else if (row < L) {
                    *reinterpret_cast<uint4 *>(o) = make_uint4(u[0], u[1], u[2], u[3]);
                    if (col + 8 < vd) *reinterpret_cast<uint4 *>(o + 8) = make_uint4(u[4], u[5], u[6], u[7]);
                }
            }
        }
        umma::fence_before();
    };

    if (warp == NS + NK) {
        // ------------------------------------------------------------ tile loads
        int issued = PER;
        bool ok = true;
        for (int c = 1; c < nc && ok; ++c) {
#pragma unroll 1
            for (int i = 0; i < PER; ++i) {
                const int x = PER * c + i;
                if (x >= RING) ok = ok && wwait(sb + B_EMPTY + 8 * (x % RING), ((x / RING) - 1) & 1, flag, a.err);
                if (!ok) break;
                tile(c, i);
                ++issued;
            }
        }
        if (!ok) {  // after an error: let the loads in flight land (bounded)
            for (int x = max(0, issued - RING); x < issued; ++x)
                umma::mbar_spin(sb + B_FULL + 8 * (x % RING), (x / RING) & 1, 4000000L);
        }
    } else if (warp == NS + NK + 1) {
        // ------------------------------------------------------------ MMAs
        constexpr bool bf = IsBf16<T>::value;
        const uint32_t i_qk = umma::idesc(128, 128, bf, false, false), i_qs = umma::idesc(128, NV, bf, false, true),
                       i_ds = umma::idesc(128, NV, bf, true, true);
        const uint32_t on = lane == 0;
        bool ok = true;
        auto full = [&](int c, int which) { return wwait(sb + B_FULL + 8 * slot_of(c, which), phase_of(c, which), flag, a.err); };
        auto wait_qk = [&](int c) {
            // (and P of the chunk before has been read: Q K^T takes its place)
            const uint32_t b = sb + B_FULL + 8 * slot_of(c, 0), f = phase_of(c, 0);
            ok = ok && __all_sync(0xffffffffu, wait_phases(b, f, sb + B_FULL + 8 * slot_of(c, KI), phase_of(c, KI), c > 0 ? sb + B_PV : b,
                                                           c > 0 ? (c - 1) & 1 : f, flag, a.err));
            umma::fence_after();
        };
        auto issue_qk = [&](int c) {
            const uint64_t dq = umma::desc(sb + slot_of(c, 0) * TILE, 16, 1024), dk = umma::desc(sb + slot_of(c, KI) * TILE, 16, 1024);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint32_t o = (uint32_t)(ks >> 2) * BLK + (uint32_t)(ks & 3) * 32u;
                if (ks < ksteps) mma_ss(on, tmem + T_QK, desc_at(dq, o), desc_at(dk, o), i_qk, ks > 0);
            }
            commit_on(on, sb + B_QK);
            if (lane == 0) mbar_arrive(sb + B_QK);  // (hands on that q and k have landed)
        };
        // one of the products of chunk c's state update: with the keys or with one of their remainders
        auto issue_ds = [&](int c, uint32_t keys, int ts, bool more) {
            const uint32_t d = tmem + T_DS - (STATES && (c & 1) ? 128 : 0);
            const uint64_t dv = umma::desc(sb + slot_of(c, VI) * TILE, BLK, 1024), dk = umma::desc(keys, BLK, 1024);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                if (ks < ts) {
                    if (ks == 0 && !bf && more) mma_ss_down(on, d, dk, dv, i_ds);
                    else mma_ss(on, d, desc_at(dk, ks * 2048u), desc_at(dv, ks * 2048u), i_ds, more || ks > 0);
                }
        };
        if (!STATES && nc > 0) {
            wait_qk(0);
            if (ok) issue_qk(0);
        }
        for (int c = 0; c < nc && ok; ++c) {
            int t, L;
            chunk(c, t, L);
            const int ts = (L + 15) / 16;
            const uint32_t kt = sb + slot_of(c, KI) * TILE, lo = sb + lo_of(c);
            const bool upd = want_end || c + 1 < nc, use_s = c > 0 || has_start;
            if (!STATES) {
                // the state's copy is there, and the accumulators of the chunk before have been read
                ok = ok && wwait(sb + B_S, c & 1, flag, a.err);
                if (!ok) break;
                umma::fence_after();
                if (use_s) {
                    const uint64_t dq = umma::desc(sb + slot_of(c, 0) * TILE, 16, 1024), ds = umma::desc(sb + S_ST, BLK, 1024);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t o = (uint32_t)(ks >> 2) * BLK + (uint32_t)(ks & 3) * 32u;
                        if (ks < ksteps) mma_ss(on, tmem + T_QS, desc_at(dq, o), desc_at(ds, ks * 2048u), i_qs, ks > 0);
                    }
                }
                commit_on(on, sb + B_EMPTY + 8 * slot_of(c, 0));
                if (MAY) commit_on(on, sb + B_QS);
                const uint32_t b = sb + B_FULL + 8 * slot_of(c, VI), f = phase_of(c, VI);
                ok = ok && __all_sync(0xffffffffu, wait_phases(sb + B_P, c & 1, b, f, b, f, flag, a.err));
                if (!ok) break;
                umma::fence_after();
                const uint64_t dv = umma::desc(sb + slot_of(c, VI) * TILE, BLK, 1024);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    if (ks < ts) mma_ts(on, tmem + T_PV, tmem + T_QK + 32 * (ks >> 1) + 8 * (ks & 1), desc_at(dv, ks * 2048u), i_qs, ks > 0);
                commit_on(on, sb + B_PV);
            } else {
                ok = ok && full(c, VI);
            }
            if (upd) {
                ok = ok && wwait(bar_of(B_K, c), par_of(c), flag, a.err);
                // (state pass: its accumulator was read, two chunks before, ahead of these keys)
                if (!ok) break;
                umma::fence_after();
                const uint32_t first = MAY && three(c) ? sb + S_ST : lo;
#pragma unroll 1
                for (uint32_t keys = first;; keys = keys != lo ? lo : kt) {
                    issue_ds(c, keys, ts, keys != first);
                    if (keys == kt) break;
                    if (keys == lo && !STATES && c + 1 < nc) wait_qk(c + 1);
                    if (!ok) break;
                }
                if (!ok) break;
                commit_on(on, bar_of(B_DS, c));
            }
            if (!ok) break;
            commit_on(on, sb + B_EMPTY + 8 * slot_of(c, KI));
            commit_on(on, sb + B_EMPTY + 8 * slot_of(c, VI));
            // (runs while the state is updated)
            if (!STATES && c + 1 < nc) issue_qk(c + 1);
        }
        // every MMA, and every arrival that waits for one, has happened before shared memory goes away
        commit_on(on, sb + B_DONE);
        umma::mbar_spin(sb + B_DONE, 0, 4000000L);
    } else if (warp >= NS) {
        // ------------------------------------------------------------ P, and the decayed keys
        const int q4 = warp & 3, row = q4 * 32 + lane;
        const uint32_t quad = tmem + ((uint32_t)(q4 * 32) << 16), swz = row & 7;
        // the i-th eight columns of this thread's row in a tile
        auto place = [&](int i) { return (uint32_t)(i >> 3) * BLK + row * 128 + (((uint32_t)(i & 7) ^ swz) << 4); };
        // zeros behind the last row of chunk c's v, as far as the MMAs read
        auto clear_v = [&](int c, int L) {
            if (!wwait(sb + B_FULL + 8 * slot_of(c, VI), phase_of(c, VI), flag, a.err)) return false;
            if (row >= L && row < (L + 15) / 16 * 16)
#pragma unroll 1
                for (int i = 0; i < 8 * vblk; ++i) umma::st_shared_v4(sb + slot_of(c, VI) * TILE + place(i), 0, 0, 0, 0);
            __syncwarp();
            return true;
        };
        // The blocks of P on the diagonal, next to it, and those that see nothing.
        auto make_p = [&](int c, int L) {
            if (!wwait(sb + B_QK, c & 1, flag, a.err)) return false;
            umma::fence_after();
            uint32_t o[16], x[32];
            float f[32];
            tld32(quad + T_QK + 32 * q4, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = reinterpret_cast<const float *>(smem + S_DIAG)[31 + lane - i];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = 0;
#pragma unroll 1
            for (int blk = rev ? 0 : q4 + 1; blk < (rev ? q4 : 4); ++blk) tst16(quad + T_QK + 32 * blk, o);
            twait32(x);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[i] = Elt<T>::pack(f[2 * i] != 0.f ? __uint_as_float(x[2 * i]) * f[2 * i] : 0.f,
                                    f[2 * i + 1] != 0.f ? __uint_as_float(x[2 * i + 1]) * f[2 * i + 1] : 0.f);
            if (rev && L < LC) {  // (a short chunk's rows see no keys behind it)
                const int most = L - 32 * q4;
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = 2 * i + 1 < most ? o[i] : 2 * i < most ? o[i] & 0xffffu : 0u;
            }
            tst16(quad + T_QK + 32 * q4, o);
            p_beyond(1, L);
            if (L < LC) {
                // the rows behind a short chunk are another sequence's: what they hold must not meet even a zero
                if (!clear_v(c, L)) return false;
                umma::fence_async_smem();
            }
            tst_wait();
            umma::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sb + B_P);
            return true;
        };
        bool ok = true;
        for (int c = 0; c < nc && ok; ++c) {
            int t, L;
            chunk(c, t, L);
            if (!STATES) {
                ok = make_p(c, L);
                // (the remainders' place: read by the update of the chunk before)
                if (want_end || c + 1 < nc) {
                    if (c > 0) ok = ok && wwait(sb + B_DS, (c - 1) & 1, flag, a.err);
                    if (three(c)) ok = ok && wwait(sb + B_QS, c & 1, flag, a.err);
                    if (ok) make_keys(c, L, 10, min(16, 8 * kblk), Int<1>());
                }
                continue;
            }
            // (half of the keys' columns, the state warps the others; the remainders' place was read two chunks before)
            ok = wwait(sb + B_FULL + 8 * slot_of(c, VI), phase_of(c, VI), flag, a.err) &&
                 wwait(sb + B_FULL + 8 * slot_of(c, KI), phase_of(c, KI), flag, a.err);
            if (ok && L < LC) clear_v(c, L);
            if (three(c) ? c >= 1 : c >= 2) ok = ok && wwait(bar_of(B_DS, three(c) ? c - 1 : c), par_of(three(c) ? c - 1 : c - 2), flag, a.err);
            if (ok) make_keys(c, L, 0, 8, Int<1>());
        }
    } else {
        // ------------------------------------------------------------ the state and the output rows
        const int q4 = warp & 3, row = q4 * 32 + lane, c0 = (warp >> 2) * CW;
        const uint32_t quad = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t tile_row = (uint32_t)(c0 >> 6) * BLK + row * 128, swz = row & 7;
        // the i-th eight of this thread's columns in a tile
        auto place = [&](int i) { return tile_row + (((uint32_t)((c0 & 63) / 8 + i) ^ swz) << 4); };
        const bool live = row < kd;
        f2 st[CW / 2];
#pragma unroll
        for (int i = 0; i < CW / 2; ++i) st[i] = 0ull;
        if (!STATES && has_start) {
            if (w.start) {
                const float *s0 = w.start + ((long long)seg.n * a.H + j) * kd * vd + (long long)row * w.rs;
#pragma unroll
                for (int i = 0; i < CW / 4; ++i) {
                    const int col = c0 + 4 * i;
                    if (!live || col >= vd) continue;
                    if (w.cs == 1) {
                        const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(s0 + col);
                        st[2 * i] = u.x, st[2 * i + 1] = u.y;
                    } else {
                        const long long cs = w.cs;
                        st[2 * i] = pack2(s0[col * cs], s0[(col + 1) * cs]), st[2 * i + 1] = pack2(s0[(col + 2) * cs], s0[(col + 3) * cs]);
                    }
                    st[2 * i] = mul2(st[2 * i], both(1.f / w.s_state)), st[2 * i + 1] = mul2(st[2 * i + 1], both(1.f / w.s_state));
                }
            }
            if (!at_start) {
                // the windows before this segment, in the walk's order
                const Cuts wc(a, a.win_len);
                int pos = rev ? seg.seq1 : seg.seq0;
                const int stop = rev ? seg.t1 : seg.t0;
                while (pos != stop) {
                    const int at = pos;
                    const int from = rev ? max(wc.last(seg, pos - 1), seg.seq0) : pos;
                    pos = rev ? from : wc.next(seg, pos);
                    const float *e = w.ext + (wc.place(seg, from) * a.H + j) * (kd * vd) + (long long)row * w.ers;
                    const f2 d = both(ex2((float)(rev ? at - from : pos - at) * lg));
#pragma unroll
                    for (int i = 0; i < CW / 2; ++i) {
                        const int col = c0 + 2 * i;
                        if (live && col < vd) st[i] = fma2(d, st[i], pack2(e[(long long)col * w.ecs], e[(long long)(col + 1) * w.ecs]));
                    }
                }
            }
        }
        uint32_t most = 0;
        auto see = [&](int i) {  // takes pair i of the state into its maximum
            float x[2];
            unpack2(st[i], x[0], x[1]);
            const uint32_t u = max(__float_as_uint(x[0]) * 2 + 0x01000000u, __float_as_uint(x[1]) * 2 + 0x01000000u);
            if (!IsBf16<T>::value && c0 + i / 4 * 8 < vd) most = max(most, u);
        };
        // the copy for chunk c
        auto put_state = [&](int c) {
            if (c0 >= NV) return true;
            f2 f = both(1.f);
            if constexpr (!IsBf16<T>::value) {
                // (columns behind vd and rows behind kd hold what was left in tensor memory and in the tile)
                const uint32_t m = __reduce_max_sync(0xffffffffu, live ? most : 0u);
                const uint32_t bar = sb + B_MAX + 8 * (warp >> 2);
                if (lane == 0) {
                    sts32(maxima(c) + 4 * (warp & 3), m);
                    mbar_arrive(bar);
                }
                if (!wwait(bar, c & 1, flag, a.err)) return false;
                f = both(two_to(copy_shift(c)));
            }
#pragma unroll
            for (int i = 0; i < CW / 8; ++i) {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = narrow2<T>(IsBf16<T>::value ? st[4 * i + e] : mul2(st[4 * i + e], f));
                umma::st_shared_v4(sb + S_ST + place(i), h[0], h[1], h[2], h[3]);
            }
            return true;
        };
        // the state after chunk c
        auto update = [&](int c, int L) {
            if (c0 >= NV) return;
            umma::fence_after();
            const f2 l1 = both(L == LC ? lds_f(sb + S_LAM) : ex2((float)L * lg)), l2 = both(L == LC ? lds_f(sb + S_LAM + 4) : 0.f);
            most = 0;
            const uint32_t at = quad + T_DS - (STATES && (c & 1) ? 128 : 0) + c0;
#pragma unroll
            for (int h = 0; h < CW / 32; ++h) {
                uint32_t x[32];
                tld32(at + 32 * h, x);
                twait32(x);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    f2 &v = st[16 * h + i];
                    v = fma2(l1, v, fma2(l2, v, f2_of(x[2 * i], x[2 * i + 1])));
                    if (!STATES) see(16 * h + i);
                }
            }
            umma::fence_before();
        };
        // The blocks of P two or three from the diagonal.
        auto make_p = [&](int c, int L) {
            if (!wwait(sb + B_QK, c & 1, flag, a.err)) return false;
            umma::fence_after();
            p_beyond(c0 ? 2 : 3, L);
            tst_wait();
            umma::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sb + B_P);
            return true;
        };
        // this warp's share of the keys: a quarter of the columns (state pass), or six and four eights of sixteen
        const int k0 = STATES ? 8 + c0 / 16 : c0 ? 6 : 0, k1 = min(STATES ? k0 + 4 : c0 ? 10 : 6, 8 * kblk);
        bool ok = true;
        if (!STATES) {
#pragma unroll
            for (int i = 0; i < CW / 2; ++i) see(i);
            ok = put_state(0);
            umma::fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(sb + B_S);
            if (ok && nc > 0) {
                int t, L;
                chunk(0, t, L);
                ok = make_p(0, L);
                if (ok && (want_end || nc > 1)) make_keys(0, L, k0, three(0) ? k0 : k1, Int<0>());
            }
        }
        int before = 0;  // (state pass) the length of the chunk before
        for (int c = 0; c < nc && ok; ++c) {
            int t, L;
            chunk(c, t, L);
            const bool upd = want_end || c + 1 < nc;
            if (STATES) {
                ok = wwait(sb + B_FULL + 8 * slot_of(c, KI), phase_of(c, KI), flag, a.err);
                if (!ok) break;
                make_keys(c, L, k0, three(c) ? k0 : k1, Int<0>());
                if (c > 0) {
                    ok = wwait(bar_of(B_DS, c - 1), par_of(c - 1), flag, a.err);
                    if (!ok) break;
                    update(c - 1, before);
                }
                before = L;
            } else {
                ok = wwait(sb + B_PV, c & 1, flag, a.err);
                if (!ok) break;
                out_rows(c, t, L, c0, c0 + 64);
                if (upd) {
                    ok = wwait(sb + B_DS, c & 1, flag, a.err);
                    if (!ok) break;
                    update(c, L);
                }
                if (c + 1 < nc) {
                    ok = put_state(c + 1);
                    if (!ok) break;
                    umma::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sb + B_S);
                    int tn, Ln;
                    chunk(c + 1, tn, Ln);
                    ok = make_p(c + 1, Ln);
                    if (ok && (want_end || c + 2 < nc)) make_keys(c + 1, Ln, k0, three(c + 1) ? k0 : k1, Int<0>());
                }
            }
        }
        if (STATES && ok && nc > 0) {
            ok = wwait(bar_of(B_DS, nc - 1), par_of(nc - 1), flag, a.err);
            if (ok) update(nc - 1, before);
        }
        if (ok && want_end && live) {
            const long long n = STATES ? (long long)(a.cu ? slot - seg.n - 1 : slot) : (long long)seg.n;  // (as `place`, which is dearer)
            float *e = STATES ? w.states + (n * a.H + j) * (kd * vd) + row : w.end + (n * a.H + j) * kd * vd + (long long)row * w.rs;
            const long long cs = STATES ? w.ecs : w.cs;
#pragma unroll
            for (int i = 0; i < CW / 4; ++i) {
                const int col = c0 + 4 * i;
                if (col >= vd) continue;
                if (!STATES) st[2 * i] = mul2(st[2 * i], both(w.s_state)), st[2 * i + 1] = mul2(st[2 * i + 1], both(w.s_state));
                if (!STATES && cs == 1) {
                    *reinterpret_cast<ulonglong2 *>(e + col) = make_ulonglong2(st[2 * i], st[2 * i + 1]);
                } else {
                    unpack2(st[2 * i], e[col * cs], e[(col + 1) * cs]);
                    unpack2(st[2 * i + 1], e[(col + 2) * cs], e[(col + 3) * cs]);
                }
            }
        }
    }
    umma::fence_before();
    __syncthreads();
    if (warp == NS + NK + 1) umma::dealloc(tmem, 512);
}

template <typename T, bool STATES, bool MAY>
cudaError_t launch_t(const LinParams &p, cudaStream_t s) {
    const long long n = lin_slots(p.a, STATES ? p.a.win_len : p.a.main_len) * p.a.H * p.a.nwalk;
    if (n == 0) return cudaSuccess;
    auto k = lin_walk_kernel<T, STATES, MAY>;
    const cudaError_t e = allow_smem(k, S_BYTES);
    if (e != cudaSuccess) return e;
    return launch_plain(k, dim3((unsigned)n), dim3(NT), S_BYTES, s, p);
}
template <bool STATES>
cudaError_t launch_any(const LinParams &p, bool bf16, cudaStream_t s) {
    bool ends = false;
    for (int i = 0; i < p.a.nwalk; ++i) ends = ends || p.w[i].end;
    if (!bf16) return launch_t<__half, STATES, false>(p, s);
    return ends ? launch_t<__nv_bfloat16, STATES, true>(p, s) : launch_t<__nv_bfloat16, STATES, false>(p, s);
}

}  // namespace

cudaError_t launch_lin_walks(const LinParams &p, bool bf16, cudaStream_t s) { return launch_any<false>(p, bf16, s); }
cudaError_t launch_lin_states(const LinParams &p, bool bf16, cudaStream_t s) { return launch_any<true>(p, bf16, s); }

}  // namespace lin
}  // namespace gdr
