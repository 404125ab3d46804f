// Selective scan for single tokens: the T tokens of every row applied one by one to its cached fp32 state, in place.
//
//   h <- exp(delta A) h + delta x B,   y = (C . h + D x) silu(z)      (delta = softplus(dt + bias) or dt + bias)
//
// Bound by HBM: 8 bytes of state a (row, channel, state) against ten of token data a (row, channel).  A channel's N
// states lie in NL = 1 .. 16 lanes side by side, four in each (one 16-byte access where N allows it), so a warp moves
// contiguous state.  A thread keeps its channel and states and walks rows of the batch, four at a time, with the states
// of the next groups on their way as asynchronous copies into shared memory that only it uses, and the next group's
// token data in registers.  The scalar work of a row (softplus, the gate) is done by one of the channel's lanes and
// handed round; the sum over the states is a butterfly over the lanes.
#include "scan.cuh"

namespace gdr {
namespace scan {
namespace {

constexpr int RB = 4;      // rows a group
constexpr int AHEAD = 2;   // groups of states in flight

// ONE: one token a row.  256 x 4096, N = 16, bf16: 32 us for 143 MB, 4.4 TB/s (65 % of a copy's rate), with 57 % of the issue
// slots taken by the states' arithmetic.  One row of 2048 channels: the launch's latency.
template <typename T, int NL, bool ONE>
__global__ void __launch_bounds__(256, 2) scan_step_kernel(const ScanArgs a, int chunk) {
    constexpr int OWN = RB > NL ? RB / NL : 1;  // rows whose scalars a lane computes (lanes past RB repeat them)
    __shared__ __align__(16) float4 ring[AHEAD][RB][256];
    const int tid = threadIdx.x, nl = tid % NL, n0 = nl * 4, lead = (tid & 31) - nl;
    const int d0 = blockIdx.x * (256 / NL) + tid / NL;
    const bool live = d0 < a.D;                          // (the others repeat the last channel and store nothing)
    const int d = live ? d0 : a.D - 1, g = d / a.Dg;
    const int b0 = blockIdx.y * chunk, b1 = min(a.B, b0 + chunk);
    const bool wide = a.st_vec && a.vec_bc, mine = n0 < a.N;
    float A2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] = n0 + i < a.N ? rate2(a.A[(long long)d * a.N + n0 + i]) : 0.f;
    const float bias = a.bias ? a.bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
    // this lane's rows of a group, and the places of the token to load next (of the first of the rows)
    const int own = RB >= NL ? nl * OWN : nl % RB, T_ = ONE ? 1 : a.T;
    const long long row0 = (long long)b0 * T_, orow = row0 + (long long)own * T_;
    const uint16_t *px = static_cast<const uint16_t *>(a.x) + orow * a.x_ld + d, *pd = static_cast<const uint16_t *>(a.dt) + orow * a.dt_ld + d;
    const uint16_t *pz = a.z ? static_cast<const uint16_t *>(a.z) + orow * a.z_ld + d : nullptr;
    const uint16_t *pb = static_cast<const uint16_t *>(a.Bm) + row0 * a.b_ld + (long long)g * a.N + n0;
    const uint16_t *pc = static_cast<const uint16_t *>(a.Cm) + row0 * a.c_ld + (long long)g * a.N + n0;
    T *py = static_cast<T *>(a.y) + orow * a.D + d;
    const long long sx = T_ * a.x_ld, sd = T_ * a.dt_ld, sz = T_ * a.z_ld, sb = T_ * a.b_ld, sc = T_ * a.c_ld, sy = (long long)T_ * a.D;
    // from a group's last token to the next group's first
    const long long gx = RB * sx - (T_ - 1) * a.x_ld, gd = RB * sd - (T_ - 1) * a.dt_ld, gz = RB * sz - (T_ - 1) * a.z_ld;
    const long long gb = RB * sb - (T_ - 1) * a.b_ld, gc = RB * sc - (T_ - 1) * a.c_ld, gy = RB * sy - (long long)(T_ - 1) * a.D;
    const long long st_step = (long long)a.D * a.N;
    float *st = a.state_out + (long long)b0 * st_step + (long long)d * a.N + n0;  // (updated in place)
    const float *next = st;                              // state to copy next

    // FULL: all rows of the group exist and every access is a whole one
    auto copy_states = [&](int b, int slot, auto full) {
#pragma unroll
        for (int r = 0; r < RB; ++r, next += st_step) {
            if (full.value) {
                if (mine) copy16(&ring[slot][r][tid], next);
            } else if (b + r < b1) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = n0 + i < a.N ? next[i] : 0.f;
                ring[slot][r][tid] = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    };
    auto copy_group = [&](int b, int slot) {
        if (wide && b + RB <= b1)
            copy_states(b, slot, Flag<true>());
        else
            copy_states(b, slot, Flag<false>());
        copies_commit();
    };
    struct Token {
        uint2 rb[RB], rc[RB];
        uint16_t x[OWN], dt[OWN], z[OWN];
    };
    auto load_token = [&](int b, Token &k, auto full) {  // of the rows from b
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            k.x[o] = k.dt[o] = k.z[o] = 0;
            if (full.value || b + own + o < b1) {
                k.x[o] = px[o * sx];
                k.dt[o] = pd[o * sd];
                if (pz) k.z[o] = pz[o * sz];
            }
        }
        const uint16_t *qb = pb, *qc = pc;
#pragma unroll
        for (int r = 0; r < RB; ++r, qb += sb, qc += sc) {
            k.rb[r] = k.rc[r] = make_uint2(0, 0);
            if (full.value) {
                if (mine) k.rb[r] = *reinterpret_cast<const uint2 *>(qb), k.rc[r] = *reinterpret_cast<const uint2 *>(qc);
            } else if (b + r < b1) {
                uint32_t v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = n0 + i < a.N ? qb[i] : 0, v[4 + i] = n0 + i < a.N ? qc[i] : 0;
                k.rb[r] = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
                k.rc[r] = make_uint2(v[4] | v[5] << 16, v[6] | v[7] << 16);
            }
        }
    };
    auto load_next = [&](int b, bool last, Token &k) {  // and on to the token after it; `last`: of its group
        if (wide && b + RB <= b1)
            load_token(b, k, Flag<true>());
        else
            load_token(b, k, Flag<false>());
        px += last ? gx : a.x_ld, pd += last ? gd : a.dt_ld, pb += last ? gb : a.b_ld, pc += last ? gc : a.c_ld;
        if (pz) pz += last ? gz : a.z_ld;
    };
    auto to_f = [](uint16_t v) { return Elt<T>::to_f(*reinterpret_cast<const T *>(&v)); };
    auto step = [&](const Token &k, float (*h)[4], int b, bool last, auto full) {
        // the scalars of this lane's rows
        float dl[OWN], u[OWN], base[OWN], gate[OWN];
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            const float x = to_f(k.x[o]), v = to_f(k.dt[o]) + bias, z = to_f(k.z[o]);
            dl[o] = a.softplus ? softplus(v) : v;
            u[o] = dl[o] * x;
            base[o] = skip * x;
            gate[o] = a.z ? z * sigmoid(z) : 1.f;
        }
        float y[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int from = lead + (RB >= NL ? r / OWN : r), o = RB >= NL ? r % OWN : 0;
            const float dr = __shfl_sync(0xffffffffu, dl[o], from), ur = __shfl_sync(0xffffffffu, u[o], from);
            float B[4], C[4];
            unpack2(widen2<T>(k.rb[r].x), B[0], B[1]);
            unpack2(widen2<T>(k.rb[r].y), B[2], B[3]);
            unpack2(widen2<T>(k.rc[r].x), C[0], C[1]);
            unpack2(widen2<T>(k.rc[r].y), C[2], C[3]);
            y[r] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[r][i] = fmaf(ex2(A2[i] * dr), h[r][i], ur * B[i]);
                y[r] = fmaf(C[i], h[r][i], y[r]);
            }
#pragma unroll
            for (int o2 = NL / 2; o2 > 0; o2 >>= 1) y[r] += __shfl_xor_sync(0xffffffffu, y[r], o2);
        }
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            float v = y[0];
#pragma unroll
            for (int e = 1; e < RB; ++e) v = e == own + o ? y[e] : v;
            if (live && nl < RB && (full.value || b + own + o < b1)) py[o * sy] = Elt<T>::from_f((base[o] + v) * gate[o]);
        }
        py += last ? gy : (long long)a.D;
    };

    Token k;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) copy_group(b0 + i * RB, i);
    load_next(b0, ONE || T_ == 1, k);
    int slot = 0;
    for (int b = b0; b < b1; b += RB) {
        copies_wait<AHEAD - 1>();
        float h[RB][4];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const float4 f = mine ? ring[slot][r][tid] : make_float4(0.f, 0.f, 0.f, 0.f);  // (padded states stay zero)
            h[r][0] = f.x, h[r][1] = f.y, h[r][2] = f.z, h[r][3] = f.w;
        }
        copy_group(b + AHEAD * RB, slot);
        slot = slot + 1 == AHEAD ? 0 : slot + 1;
        const bool full = wide && b + RB <= b1;
        for (int t = 0; t < T_; ++t) {
            const Token now = k;
            const bool last = ONE || t + 1 == T_;
            if (!last)
                load_next(b, t + 2 == T_, k);
            else if (b + RB < b1)
                load_next(b + RB, ONE || T_ == 1, k);
            if (full)
                step(now, h, b, last, Flag<true>());
            else
                step(now, h, b, last, Flag<false>());
        }
#pragma unroll
        for (int r = 0; r < RB; ++r, st += st_step) {
            if (full) {
                if (live && mine) *reinterpret_cast<float4 *>(st) = make_float4(h[r][0], h[r][1], h[r][2], h[r][3]);
            } else if (live && b + r < b1) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n0 + i < a.N) st[i] = h[r][i];
            }
        }
    }
    copies_wait<0>();
}

template <typename T>
cudaError_t launch_t(const ScanArgs &a, int L, cudaStream_t s) {
    const bool one = a.T == 1;
    const int per = 256 / L, xb = (a.D + per - 1) / per;
    // Rows a block: as many as leave four blocks an SM, of which two are resident at a time, so that a thread's fixed work is
    // shared by the rows.
    const long long most = (long long)a.B * xb / (4 * kSMs);
    int chunk = (int)(most / RB * RB);
    chunk = chunk < RB ? RB : chunk > 64 ? 64 : chunk;
    if ((a.B + chunk - 1) / chunk > 65535) chunk = ((a.B + 65534) / 65535 + RB - 1) / RB * RB;
    const dim3 grid((unsigned)xb, (unsigned)((a.B + chunk - 1) / chunk)), block(256);
    switch (L) {
        case 1: return one ? launch_plain(scan_step_kernel<T, 1, true>, grid, block, 0, s, a, chunk) : launch_plain(scan_step_kernel<T, 1, false>, grid, block, 0, s, a, chunk);
        case 2: return one ? launch_plain(scan_step_kernel<T, 2, true>, grid, block, 0, s, a, chunk) : launch_plain(scan_step_kernel<T, 2, false>, grid, block, 0, s, a, chunk);
        case 4: return one ? launch_plain(scan_step_kernel<T, 4, true>, grid, block, 0, s, a, chunk) : launch_plain(scan_step_kernel<T, 4, false>, grid, block, 0, s, a, chunk);
        case 8: return one ? launch_plain(scan_step_kernel<T, 8, true>, grid, block, 0, s, a, chunk) : launch_plain(scan_step_kernel<T, 8, false>, grid, block, 0, s, a, chunk);
        default: return one ? launch_plain(scan_step_kernel<T, 16, true>, grid, block, 0, s, a, chunk) : launch_plain(scan_step_kernel<T, 16, false>, grid, block, 0, s, a, chunk);
    }
}

}  // namespace

cudaError_t launch_scan_step(const ScanArgs &a, int L, bool bf16, cudaStream_t s) {
    return bf16 ? launch_t<__nv_bfloat16>(a, L, s) : launch_t<__half>(a, L, s);
}

}  // namespace scan
}  // namespace gdr
