// The GDN layer over drafted tokens: the short conv and the delta rule along a
// chain or a tree of up to 64 tokens of each sequence, which leave the held
// state alone, and the commit of the accepted path into it.
//
// The recurrence along the path to token i, S_i = a_i S_p (I - b_i k_i k_i^T) +
// b_i v_i k_i^T with p its parent, is S_i = a_i S_p + u_i k_i^T for u_i = b_i
// (v_i - a_i S_p k_i).  With g_i the sum of log a over i and its ancestors,
//     u_i = b_i (v_i - e^{g_i} S_0 k_i - sum_{j anc i} e^{g_i - g_j} (k_j . k_i) u_j)
//     o_i = S_i q_i = e^{g_i} S_0 q_i + sum_{j anc i, i} e^{g_i - g_j} (k_j . q_i) u_j
// so no state but S_0 is formed, S_0 is read once for all tokens of the
// sequence, and the state after any token n follows from the u:
//     S_n = e^{g_n} S_0 + sum_{j anc n, n} e^{g_n - g_j} u_j k_j^T.
#include "drafts.cuh"

namespace gdn {

static __device__ int g_draft_error;      // a value beyond fp16; debug: a store's index
static __device__ int g_draft_skipped;    // an offset or node of the caller's, out of range

constexpr float LOG_A_MIN = -1.0e4f;      // e^-10000 is 0 in fp32, and sums of it stay finite (a = 0: log a = -inf)

// ------------------------------------------------------------ conv

struct ConvTreeArgs {
    DraftTokens d;
    const uint16_t* qkvz;
    int64_t ld_qkvz;
    const float* ba;
    int64_t ld_ba;
    const float* tail;     // [n_seqs][c_conv][3]
    const float* conv_w;   // [c_conv][4]
    const float* A_log;
    const float* dt_bias;
    uint16_t* out;         // fp16 [n_tokens][c_conv]
    float* log_a;
    float* b;
    int c_conv, n_heads, n_qk_norm, n_q, hv, head_blocks;
    float eps, q_scale;
};

constexpr int CT_WARPS = 8;
constexpr int CT_TOKENS = 8;

// Block (token run, head group, sequence): a warp per head.  The last slice of
// y computes the gates.
template <int CPL>
__global__ void __launch_bounds__(CT_WARPS * 32) conv_tree_kernel(const __grid_constant__ ConvTreeArgs a) {
    constexpr int D = CPL * 32;
    const int s = blockIdx.z;
    int first;
    const int n = draft_range(a.d, s, first, g_draft_skipped);
    const int i0 = blockIdx.x * CT_TOKENS, i1 = min(n, i0 + CT_TOKENS);
    if (i0 >= i1) return;
    if (static_cast<int>(blockIdx.y) == a.head_blocks) {
        for (int e = threadIdx.x; e < (i1 - i0) * a.hv; e += blockDim.x) {
            const int64_t t = first + i0 + e / a.hv;
            const int h = e % a.hv;
            gate_values(a.ba[t * a.ld_ba + h], a.ba[t * a.ld_ba + a.hv + h], a.A_log[h], a.dt_bias[h], a.log_a[t * a.hv + h],
                        a.b[t * a.hv + h]);
        }
        return;
    }
    const int head = blockIdx.y * CT_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (head >= a.n_heads) return;
    const int c0 = head * D + lane * CPL;
    const bool norm = head < a.n_qk_norm;
    for (int i = i0; i < i1; ++i) {
        // the token, its parent, grandparent and great-grandparent; -1, -2, -3 are the conv state from its newest entry on
        int at[4];
        at[3] = i;
#pragma unroll
        for (int m = 2; m >= 0; --m) at[m] = at[m + 1] < 0 ? at[m + 1] - 1 : draft_parent(draft_ancestors(a.d, first, at[m + 1]));
        float y[CPL], ss = 0.0f;
#pragma unroll
        for (int e = 0; e < CPL; ++e) {
            const int c = c0 + e;
            float x[4];
#pragma unroll
            for (int m = 0; m < 4; ++m)
                x[m] = at[m] < 0 ? a.tail[(static_cast<int64_t>(s) * a.c_conv + c) * 3 + 3 + at[m]]
                                 : bf16_bits_to_float(a.qkvz[static_cast<int64_t>(first + at[m]) * a.ld_qkvz + c]);
            const float4 w = *reinterpret_cast<const float4*>(a.conv_w + static_cast<int64_t>(c) * 4);
            y[e] = conv4_silu(w, x[0], x[1], x[2], x[3]);
            ss = fmaf(y[e], y[e], ss);
        }
        if (norm) {
            ss = warp_sum(ss);
            const float r = rsqrtf(ss + a.eps) * (head < a.n_q ? a.q_scale : 1.0f);
#pragma unroll
            for (int e = 0; e < CPL; ++e) y[e] *= r;
        }
        uint16_t* dst = a.out + static_cast<int64_t>(first + i) * a.c_conv + c0;
        bool over = norm && !(ss <= 3.0e38f);
#pragma unroll
        for (int e = 0; e < CPL; ++e) {
            over |= !(fabsf(y[e]) <= 65504.0f);
            if (GDN_IN_RANGE(g_draft_error, first + i < a.d.n_tokens && c0 + e < a.c_conv)) dst[e] = __half_as_ushort(__float2half_rn(y[e]));
        }
        if (over) atomicCAS(&g_draft_error, 0, static_cast<int>(ERR_RANGE));
    }
}

cudaError_t launch_conv_tree(const gdn_layer& L, const DraftTokens& d, const uint16_t* qkvz, int64_t ld_qkvz, const float* ba, int64_t ld_ba,
                             const float* tail, uint16_t* out, float* log_a, float* b, cudaStream_t st) {
    ConvTreeArgs a;
    a.d = d;
    a.qkvz = qkvz;
    a.ld_qkvz = ld_qkvz;
    a.ba = ba;
    a.ld_ba = ld_ba;
    a.tail = tail;
    a.conv_w = L.conv_w;
    a.A_log = L.A_log;
    a.dt_bias = L.dt_bias;
    a.out = out;
    a.log_a = log_a;
    a.b = b;
    a.n_heads = 2 * L.n_qk_heads + L.n_v_heads;
    a.c_conv = a.n_heads * L.dk;
    a.n_qk_norm = 2 * L.n_qk_heads;
    a.n_q = L.n_qk_heads;
    a.hv = L.n_v_heads;
    a.head_blocks = (a.n_heads + CT_WARPS - 1) / CT_WARPS;
    a.eps = L.eps_l2;
    a.q_scale = L.q_scale;
    const dim3 grid((d.max_new + CT_TOKENS - 1) / CT_TOKENS, a.head_blocks + (L.gate_log_a ? 0 : 1), d.n_seqs);
    if (L.dk == 128)
        conv_tree_kernel<4><<<grid, CT_WARPS * 32, 0, st>>>(a);
    else
        conv_tree_kernel<2><<<grid, CT_WARPS * 32, 0, st>>>(a);
    return cudaGetLastError();
}

// ------------------------------------------------------------ delta rule

struct DeltaTreeArgs {
    DraftTokens d;
    const uint16_t* qkv;   // fp16 [n_tokens][c_conv]
    const float* log_a;    // [n_tokens][hv]
    const float* b;
    const float* state;    // [n_seqs][hv][D][D]
    uint16_t* o;           // fp16 [n_tokens][hv][D]
    float* delta;          // [n_tokens][hv][D]
    int hv, ratio, c_qk, c_conv;
};

__device__ __forceinline__ float clamp_log_a(float la) { return la < LOG_A_MIN ? LOG_A_MIN : la; }

template <int D>
struct DeltaTreeSmem {
    float k[GDN_MAX_NEW][D], q[GDN_MAX_NEW][D], u[GDN_MAX_NEW][D], o[GDN_MAX_NEW][D];
    float kk[GDN_MAX_NEW][GDN_MAX_NEW], qk[GDN_MAX_NEW][GDN_MAX_NEW];
    double g[GDN_MAX_NEW];
    uint64_t anc[GDN_MAX_NEW];
    float la[GDN_MAX_NEW], b[GDN_MAX_NEW];
};

// One CTA per (value head, sequence), a thread per state row.
template <int D>
__global__ void __launch_bounds__(D) delta_tree_kernel(const __grid_constant__ DeltaTreeArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    DeltaTreeSmem<D>& sm = *reinterpret_cast<DeltaTreeSmem<D>*>(raw);
    const int h = blockIdx.x, s = blockIdx.y, hk = h / a.ratio, tid = threadIdx.x;
    int first;
    const int n = draft_range(a.d, s, first, g_draft_skipped);
    if (n == 0) return;
    for (int e = tid; e < n; e += D) {
        sm.anc[e] = draft_ancestors(a.d, first, e);
        sm.la[e] = clamp_log_a(a.log_a[static_cast<int64_t>(first + e) * a.hv + h]);
        sm.b[e] = a.b[static_cast<int64_t>(first + e) * a.hv + h];
    }
    for (int i = 0; i < n; ++i) {
        const uint16_t* row = a.qkv + static_cast<int64_t>(first + i) * a.c_conv;
        sm.q[i][tid] = __half2float(__ushort_as_half(row[hk * D + tid]));
        sm.k[i][tid] = __half2float(__ushort_as_half(row[a.c_qk + hk * D + tid]));
        sm.u[i][tid] = __half2float(__ushort_as_half(row[2 * a.c_qk + h * D + tid]));
    }
    __syncthreads();
    for (int i = tid; i < n; i += D) {
        double g = sm.la[i];
        for (uint64_t m = sm.anc[i]; m; m &= m - 1) g += sm.la[__ffsll(static_cast<long long>(m)) - 1];
        sm.g[i] = g;
    }
    __syncthreads();
    for (int e = tid; e < n * n; e += D) {
        const int i = e / n, j = e % n;
        if (j != i && !(sm.anc[i] >> j & 1)) continue;
        float kk = 0.0f, qk = 0.0f;
        for (int c = 0; c < D; ++c) {
            kk = fmaf(sm.k[j][c], sm.k[i][c], kk);
            qk = fmaf(sm.k[j][c], sm.q[i][c], qk);
        }
        const float w = expf(static_cast<float>(sm.g[i] - sm.g[j]));
        sm.kk[i][j] = w * kk;
        sm.qk[i][j] = w * qk;
    }
    const float* row = a.state + ((static_cast<int64_t>(s) * a.hv + h) * D + tid) * D;
    for (int i = 0; i < n; ++i) {
        float sk = 0.0f, sq = 0.0f;
        for (int c = 0; c < D; ++c) {
            sk = fmaf(row[c], sm.k[i][c], sk);
            sq = fmaf(row[c], sm.q[i][c], sq);
        }
        const float w = expf(static_cast<float>(sm.g[i]));
        sm.u[i][tid] -= w * sk;
        sm.o[i][tid] = w * sq;
    }
    __syncthreads();
    bool over = false;
    for (int i = 0; i < n; ++i) {
        float u = sm.u[i][tid], o = sm.o[i][tid];
        for (uint64_t m = sm.anc[i]; m; m &= m - 1) {
            const int j = __ffsll(static_cast<long long>(m)) - 1;
            u = fmaf(-sm.kk[i][j], sm.u[j][tid], u);
            o = fmaf(sm.qk[i][j], sm.u[j][tid], o);
        }
        u *= sm.b[i];
        o = fmaf(sm.qk[i][i], u, o);
        sm.u[i][tid] = u;
        over |= !(fabsf(o) <= 65504.0f);
        const int64_t at = (static_cast<int64_t>(first + i) * a.hv + h) * D + tid;
        if (GDN_IN_RANGE(g_draft_error, first + i < a.d.n_tokens)) {
            a.delta[at] = u;
            a.o[at] = __half_as_ushort(__float2half_rn(o));
        }
    }
    if (over) atomicCAS(&g_draft_error, 0, static_cast<int>(ERR_RANGE));
}

template <int D>
static cudaError_t delta_tree_launch(const DeltaTreeArgs& a, cudaStream_t st) {
    static PerDeviceOnce once;
    once.run([](int) {
        cudaFuncSetAttribute(delta_tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(DeltaTreeSmem<D>));
    });
    delta_tree_kernel<D><<<dim3(a.hv, a.d.n_seqs), D, sizeof(DeltaTreeSmem<D>), st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_delta_tree(const gdn_layer& L, const DraftTokens& d, const uint16_t* qkv, const float* log_a, const float* b,
                              const float* state, uint16_t* o, float* delta, cudaStream_t st) {
    DeltaTreeArgs a;
    a.d = d;
    a.qkv = qkv;
    a.log_a = log_a;
    a.b = b;
    a.state = state;
    a.o = o;
    a.delta = delta;
    a.hv = L.n_v_heads;
    a.ratio = L.n_v_heads / L.n_qk_heads;
    a.c_qk = L.n_qk_heads * L.dk;
    a.c_conv = 2 * a.c_qk + L.n_v_heads * L.dv;
    return L.dk == 128 ? delta_tree_launch<128>(a, st) : delta_tree_launch<64>(a, st);
}

// ------------------------------------------------------------ commit

struct CommitArgs {
    DraftTokens d;
    const uint16_t* qkv;
    const float* log_a;
    const float* delta;
    const int32_t* node;     // [n_seqs], -1: nothing accepted
    const float* state_in;
    float* state_out;
    const uint16_t* qkvz;    // null: no conv state
    int64_t ld_qkvz;
    const float* tail_in;
    float* tail_out;
    int hv, ratio, c_qk, c_conv;
};

constexpr int CM_THREADS = 256;

// The accepted token of sequence s, -1 where there is none; n: its tokens.
__device__ __forceinline__ int commit_node(const CommitArgs& a, int s, int n) {
    const int node = a.node[s];
    if (node >= -1 && node < n) return node;
    atomicCAS(&g_draft_skipped, 0, static_cast<int>(ERR_INDEX));
    return -1;
}

// Block (value head, sequence): the head's state; blocks past the heads: the conv state of CM_THREADS channels.
template <int D>
__global__ void __launch_bounds__(CM_THREADS) commit_kernel(const __grid_constant__ CommitArgs a) {
    extern __shared__ float cm[];                      // k [path][D], u [path][D]
    __shared__ int path[GDN_MAX_NEW];
    __shared__ float w[GDN_MAX_NEW];
    __shared__ float la[GDN_MAX_NEW];
    __shared__ float grow;
    const int s = blockIdx.y, tid = threadIdx.x;
    int first;
    const int n = draft_range(a.d, s, first, g_draft_skipped);
    const int node = commit_node(a, s, n);
    if (static_cast<int>(blockIdx.x) >= a.hv) {
        const int c = (blockIdx.x - a.hv) * CM_THREADS + tid;
        if (c >= a.c_conv) return;
        const float* in = a.tail_in + (static_cast<int64_t>(s) * a.c_conv + c) * 3;
        float x[3];
        int at = node;
#pragma unroll
        for (int m = 2; m >= 0; --m) {
            // at: a token, or -1, -2, -3: the old state from its newest entry on
            x[m] = at < 0 ? in[3 + at] : bf16_bits_to_float(a.qkvz[static_cast<int64_t>(first + at) * a.ld_qkvz + c]);
            at = at < 0 ? at - 1 : draft_parent(draft_ancestors(a.d, first, at));
        }
        float* out = a.tail_out + (static_cast<int64_t>(s) * a.c_conv + c) * 3;
#pragma unroll
        for (int m = 0; m < 3; ++m) out[m] = x[m];
        return;
    }
    const int h = blockIdx.x, hk = h / a.ratio;
    const uint64_t on = node < 0 ? 0ull : draft_ancestors(a.d, first, node) | 1ull << node;
    const int np = __popcll(on);
    for (int j = tid; j < n; j += CM_THREADS)
        if (on >> j & 1) {
            const int at = __popcll(on & ((1ull << j) - 1));
            path[at] = j;
            la[at] = clamp_log_a(a.log_a[static_cast<int64_t>(first + j) * a.hv + h]);
        }
    __syncthreads();
    for (int j = tid; j <= np; j += CM_THREADS) {      // entry j - 1's decay: what follows it; all of it: the state's
        double g = 0.0;
        for (int m = j; m < np; ++m) g += la[m];
        const float e = expf(static_cast<float>(g));
        if (j == 0) grow = e;
        else w[j - 1] = e;
    }
    __syncthreads();
    float* ks = cm;
    float* us = cm + np * D;
    for (int e = tid; e < np * D; e += CM_THREADS) {
        const int64_t t = first + path[e / D];
        ks[e] = __half2float(__ushort_as_half(a.qkv[t * a.c_conv + a.c_qk + hk * D + e % D]));
        us[e] = w[e / D] * a.delta[(t * a.hv + h) * D + e % D];
    }
    __syncthreads();
    const int64_t base = (static_cast<int64_t>(s) * a.hv + h) * D * D;
    for (int e = 4 * tid; e < D * D; e += 4 * CM_THREADS) {
        float4 v = *reinterpret_cast<const float4*>(a.state_in + base + e);
        if (np) {
            v.x *= grow; v.y *= grow; v.z *= grow; v.w *= grow;
        }
        for (int j = 0; j < np; ++j) {
            const float u = us[j * D + e / D];
            const float4 k = *reinterpret_cast<const float4*>(ks + j * D + e % D);
            v.x = fmaf(u, k.x, v.x); v.y = fmaf(u, k.y, v.y); v.z = fmaf(u, k.z, v.z); v.w = fmaf(u, k.w, v.w);
        }
        *reinterpret_cast<float4*>(a.state_out + base + e) = v;
    }
}

template <int D>
static cudaError_t commit_launch(const CommitArgs& a, cudaStream_t st) {
    constexpr int SMEM = 2 * GDN_MAX_NEW * D * 4;
    static PerDeviceOnce once;
    once.run([](int) { cudaFuncSetAttribute(commit_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM); });
    const int conv_blocks = a.qkvz ? (a.c_conv + CM_THREADS - 1) / CM_THREADS : 0;
    commit_kernel<D><<<dim3(a.hv + conv_blocks, a.d.n_seqs), CM_THREADS, 2 * a.d.max_new * D * 4, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_delta_commit(const gdn_layer& L, const DraftTokens& d, const uint16_t* qkv, const float* log_a, const float* delta,
                                const int32_t* node, const float* state_in, float* state_out, const uint16_t* qkvz, int64_t ld_qkvz,
                                const float* tail_in, float* tail_out, cudaStream_t st) {
    CommitArgs a;
    a.d = d;
    a.qkv = qkv;
    a.log_a = log_a;
    a.delta = delta;
    a.node = node;
    a.state_in = state_in;
    a.state_out = state_out;
    a.qkvz = qkvz;
    a.ld_qkvz = ld_qkvz;
    a.tail_in = tail_in;
    a.tail_out = tail_out;
    a.hv = L.n_v_heads;
    a.ratio = L.n_v_heads / L.n_qk_heads;
    a.c_qk = L.n_qk_heads * L.dk;
    a.c_conv = 2 * a.c_qk + L.n_v_heads * L.dv;
    return L.dk == 128 ? commit_launch<128>(a, st) : commit_launch<64>(a, st);
}

int* draft_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_draft_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

int* draft_skipped_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_draft_skipped) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace gdn
