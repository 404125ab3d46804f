// What the linear attention's entry points and its kernels share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "host.h"

namespace gdr {
namespace lin {

constexpr int LC = 128;               // tokens a chunk
constexpr int LD = 128;               // the largest head dim: the tiles' width

// One walk over the tokens,  out_r = s_out (sum over s <= r of s_kv lambda^(r-s) (q_r . k_s) v_s + the start's part),
// or backwards in time (s >= r).  Forward: (q, k, v) -> o.  Backward: (do, v, k) -> dq, and backwards in time
// (v, do, q) -> dk and (k, q, do) -> dv.
struct Walk {
    CUtensorMap tq, tk, tv;  // [tokens][heads][cols], boxes 64 x 1 x 128; tq, tk have kd columns, tv vd
    int kd, vd;
    int q_div, k_div, v_div; // head of the tensor = walk's head / div
    bool rev;
    float s_kv, s_out;
    float s_state, s_key;    // s_kv = s_state s_key; the states inside are 1 / s_state, a power of two, of the formula's
    const float *start;      // states before the walk's first token (rev: gradients behind the last), or null
    float *end;              // states behind its last token (rev: gradients before the first), or null
    int rs, cs;              // element (row of kd, column of vd) of start and end: row * rs + column * cs
    const float *ext;        // the windows' own end states, [place][H][kd x vd], element row * ers + column * ecs
    int ers, ecs;
    float *states;           // the state pass' output: those states, element column * ecs + row
    void *out;               // [tokens][H][vd], 16-bit or fp32
    bool out_f32;
};

struct LinArgs {
    const float *decay;      // [H], log decay a token
    int B, T, H, N;          // N sequences
    const int32_t *cu;       // packed: [N + 1]; null: dense rows
    unsigned *err;
    int main_len, win_len;   // tokens of a segment, and of the windows whose states are summed up for its start
    int nwalk;
};

constexpr int kMaxWalks = 3;
struct LinParams {
    Walk w[kMaxWalks];
    LinArgs a;
};

// Places of a launch: every sequence is cut at the multiples of len (dense: of its row; packed: of the token axis).
inline long long lin_slots(const LinArgs &a, int len) {
    const long long per = (a.T + (long long)len - 1) / len;
    return a.cu ? a.N + per : (long long)a.N * (per > 0 ? per : 1);
}

// Exchanged states of a walk and head: one of every interval of len tokens.
inline long long lin_places(const LinArgs &a, int len) { return (a.T + (long long)len - 1) / len * (a.cu ? 1 : a.N); }

cudaError_t launch_lin_walks(const LinParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_lin_states(const LinParams &p, bool bf16, cudaStream_t s);

// Sums of group neighbouring heads: part [rows, H, D] fp32 -> out [rows, H / group, D].
cudaError_t launch_lin_group_sum(const float *part, void *out, long long rows, int heads, int group, int D, bool bf16,
                                 cudaStream_t s);

struct StepArgs {
    const void *q, *k, *v;
    const float *decay;
    float *state;
    void *o;
    long long q_ld, k_ld, v_ld;
    int B, T, Hk, H, K, V;
    float scale;
};
cudaError_t launch_lin_step(const StepArgs &a, bool bf16, cudaStream_t s);

}  // namespace lin
}  // namespace gdr
