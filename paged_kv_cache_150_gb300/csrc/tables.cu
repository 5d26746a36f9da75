// A step's tables on the GPU (pa_extend_tables, pa_release_tables): blocks for
// the new tokens of a batch of requests taken off a free stack, its block
// tables, lengths, row offsets and slot map; and blocks given back.
//
// With L_i tokens before the step and n_i new ones, block size B:
//   request i takes ceil((L_i + n_i) / B) - ceil(L_i / B) blocks, whose place on
//   the stack is an exclusive prefix sum over the requests; token t of it has the
//   slot table[p / B] * B + p % B, p = L_i + t.
// Two kernels: one CTA checks every request and scans (a call that cannot be
// met changes nothing, so nothing is written before the last check), then a
// grid of (request, slice) CTAs fills tables and slots.  Slots of new blocks
// are read off the stack, not off the table entries that the same kernel
// writes, so its CTAs do not depend on one another.  Everything is int32 and a
// call moves some bytes per request beside the table rows: it is bound by the
// two launches' latency until the tables reach megabytes.
#include "prefill_plan.cuh"  // block_scan_1024

namespace pa {

// One request as the fill kernels see it (16 bytes, one load).
struct __align__(16) TableReq {
    int32_t row;    // row of the tables, -1: none
    int32_t old;    // tokens before the step
    int32_t len;    // tokens after it
    int32_t first;  // place of its first block: below the stack's top, or above its count (release)
};

struct TablesArgs {
    int32_t *tables;
    const int32_t *lens;
    int32_t *lens_out;
    int32_t *free_list;
    const int32_t *free_count;
    int32_t *free_count_out;
    int32_t R, W, NB, B;
    const int32_t *rows, *new_lens;
    int32_t N;
    int32_t *batch_tables;
    int32_t BW;  // its width
    int32_t *seq_lens, *cu_q, *slots;
    int32_t max_tokens;
    TableReq *reqs;   // [N]
    int32_t *claims;  // [R] the request that names each row
    int32_t *ctl;     // [0] the stack's count when the call began
    unsigned int *err;
};

__device__ __forceinline__ int32_t blocks_of(int32_t tokens, int32_t B) {
    return (int32_t)(((int64_t)tokens + B - 1) / B);
}

// Row of request i, -1 if there is none such.
__device__ __forceinline__ int32_t row_of(const TablesArgs &a, int32_t i) {
    const int32_t r = a.rows ? a.rows[i] : i;
    return r >= 0 && r < a.R ? r : -1;
}

// Whether request i is the one that its row was claimed for (of the requests
// that name one row, one is: the others refuse the call).
__device__ __forceinline__ bool owns_row(const TablesArgs &a, int32_t i, int32_t row) {
    return !a.rows || a.claims[row] == i;
}

// Sum of x over 1024 threads in 64 bits (every thread gets it).
__device__ __forceinline__ int64_t block_sum_1024(int64_t x, int64_t *warp_sums) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();  // the previous sum's reads
    if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = x;
    __syncthreads();
    x = warp_sums[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Checks and prefix sums of a call.  kRelease: the requests give back all their
// blocks; else they take blocks for their new tokens.
template <bool kRelease>
__global__ void __launch_bounds__(1024) tables_plan_kernel(const __grid_constant__ TablesArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ int32_t warp_incl[32];
    __shared__ int64_t warp_sums[32];
    const int tid = threadIdx.x;
    const int64_t max_len = (int64_t)a.W * a.B;
    const int32_t count = *a.free_count;
    if (a.rows) {
        for (int32_t i = tid; i < a.N; i += 1024) {
            const int32_t row = row_of(a, i);
            if (row >= 0) a.claims[row] = i;
        }
        __syncthreads();
    }
    // Requests may be many: what a thread finds out about its own is worked
    // out again in the second pass.
    struct Look {
        int32_t row, old, len, blocks;  // blocks taken or given back
        unsigned int bad;
    };
    auto look = [&](int32_t i) {
        Look q{row_of(a, i), 0, 0, 0, 0u};
        if (q.row < 0 || !owns_row(a, i, q.row)) {
            q.bad = kErrBounds;
            q.row = -1;
            return q;
        }
        const int32_t old = a.lens[q.row];
        if (old < 0 || old > max_len) {
            q.bad = kErrLength;
            return q;
        }
        q.old = q.len = old;
        if (kRelease) {
            q.blocks = blocks_of(old, a.B);
            return q;
        }
        const int32_t n = a.new_lens[i];
        if (n < 0 || (int64_t)old + n > max_len) {
            q.bad = kErrLength;
            return q;
        }
        q.len = old + n;
        q.blocks = blocks_of(q.len, a.B) - blocks_of(old, a.B);
        if (a.batch_tables && blocks_of(q.len, a.B) > a.BW) q.bad = kErrBounds;
        return q;
    };
    unsigned int bad = count < 0 || count > a.NB ? kErrBounds : 0u;
    int64_t blocks = 0, tokens = 0;
    Look mine{-1, 0, 0, 0, 0u};
    for (int32_t i = tid; i < a.N; i += 1024) {
        const Look q = look(i);
        if (i == tid) mine = q;
        bad |= q.bad;
        blocks += q.blocks;
        tokens += q.len - q.old;
    }
    blocks = block_sum_1024(blocks, warp_sums);
    tokens = kRelease ? 0 : block_sum_1024(tokens, warp_sums);
    bad = (__syncthreads_or((int)(bad & kErrBounds)) ? kErrBounds : 0u) | (__syncthreads_or((int)(bad & kErrLength)) ? kErrLength : 0u);
    if (kRelease) {
        if (!bad && count + blocks > a.NB) bad = kErrBounds;  // more blocks than the pool has
    } else if (!bad) {
        if (tokens > a.max_tokens)
            bad = kErrBounds;
        else if (blocks > count)
            bad = kErrNoBlocks;
    }
    const bool ok = bad == 0;
    int32_t at = 0, cu = 0;
    for (int32_t base = 0; base < a.N; base += 1024) {
        const int32_t i = base + tid;
        Look q{-1, 0, 0, 0, 0u};
        if (i < a.N) q = base == 0 ? mine : look(i);
        if (!ok) q.blocks = 0, q.len = q.old;
        int32_t total;
        const int32_t incl = block_scan_1024(q.blocks, at, warp_incl, &total);
        at = total;
        if (i < a.N) a.reqs[i] = TableReq{ok || !kRelease ? q.row : -1, q.old, q.len, incl - q.blocks};
        if (!kRelease) {
            const int32_t n = q.len - q.old;
            const int32_t cu_incl = block_scan_1024(n, cu, warp_incl, &total);
            cu = total;
            if (i < a.N) {
                a.cu_q[i] = cu_incl - n;
                a.seq_lens[i] = q.len;
            }
        }
    }
    if (tid == 0) {
        if (!kRelease) a.cu_q[a.N] = cu;
        a.ctl[0] = count;
        *a.free_count_out = kRelease ? count + at : count - at;
        if (!ok) atomicOr(a.err, bad);
    }
    // The lengths: last, as lens_out may be lens.
    if (a.lens_out != a.lens) {
        for (int32_t r = tid; r < a.R; r += 1024) a.lens_out[r] = a.lens[r];
        __syncthreads();
    }
    if (ok) {
        for (int32_t i = tid; i < a.N; i += 1024) {
            const TableReq q = a.reqs[i];  // this thread's own
            a.lens_out[q.row] = kRelease ? 0 : q.len;
        }
    }
}

// Tables and slots: CTA (i, y) takes the y-th part of request i's.
__global__ void __launch_bounds__(256) extend_fill_kernel(const __grid_constant__ TablesArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t i = blockIdx.x;
    const int32_t tid = blockIdx.y * 256 + threadIdx.x, stride = gridDim.y * 256;
    const int32_t total = a.cu_q[a.N];
    // rows of the slot map behind the last token
    for (int64_t t = (int64_t)total + (int64_t)i * stride + tid; t < a.max_tokens; t += (int64_t)gridDim.x * stride) a.slots[t] = -1;
    if (i >= a.N) return;
    const TableReq q = a.reqs[i];
    const int32_t cu = a.cu_q[i], top = a.ctl[0] - 1 - q.first;  // the stack's place of its first new block
    const int32_t nb0 = blocks_of(q.old, a.B), nb1 = blocks_of(q.len, a.B);
    int32_t *row = a.tables + (int64_t)max(q.row, 0) * a.W;
    if (a.batch_tables) {
        int32_t *out = a.batch_tables + (int64_t)i * a.BW;
        const int32_t held = q.row < 0 ? 0 : min(nb0, a.BW);
        for (int32_t j = tid; j < a.BW; j += stride) {
            int32_t b = -1;
            if (j < held) {
                b = row[j];
            } else if (j < nb1) {
                b = a.free_list[top - (j - nb0)];
                row[j] = b;
            }
            out[j] = b;
        }
    } else {
        for (int32_t j = nb0 + tid; j < nb1; j += stride) row[j] = a.free_list[top - (j - nb0)];
    }
    for (int32_t t = tid; t < q.len - q.old; t += stride) {
        const int32_t p = q.old + t, j = p / a.B;
        const int32_t b = j < nb0 ? row[j] : a.free_list[top - (j - nb0)];
        const bool good = b >= 0 && b < a.NB;
        if (!good) atomicOr(a.err, kErrBounds);
        a.slots[cu + t] = good ? b * a.B + (p - j * a.B) : -1;
    }
}

// The blocks of CTA (i, y)'s part of request i onto the stack.
__global__ void __launch_bounds__(256) release_fill_kernel(const __grid_constant__ TablesArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const TableReq q = a.reqs[blockIdx.x];
    if (q.row < 0) return;
    const int32_t nb = blocks_of(q.old, a.B), at = a.ctl[0] + q.first;
    const int32_t *row = a.tables + (int64_t)q.row * a.W;
    for (int32_t j = blockIdx.y * 256 + threadIdx.x; j < nb; j += gridDim.y * 256) {
        const int32_t b = row[j];
        if (b < 0 || b >= a.NB) atomicOr(a.err, kErrBounds);
        a.free_list[at + j] = b;
    }
}

namespace {

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t tables_workspace(int32_t N, int32_t R) {
    return 256 + align256(sizeof(TableReq) * (size_t)std::max(N, 1)) + align256(sizeof(int32_t) * (size_t)R);
}

// Checks of both calls; fills in a.
pa_status_t tables_args(const pa_tables_t *s, const int32_t *rows, int32_t N, void *workspace, size_t workspace_bytes,
                        TablesArgs *a) {
    if (!s || N < 0) return PA_ERR_INVALID_ARG;
    if (s->num_rows <= 0 || s->max_blocks_per_row <= 0 || s->num_blocks <= 0 || s->block_size <= 0) return PA_ERR_INVALID_ARG;
    if ((int64_t)s->num_rows * s->max_blocks_per_row >= ((int64_t)1 << 31) ||
        (int64_t)s->max_blocks_per_row * s->block_size >= ((int64_t)1 << 31) ||
        (int64_t)s->num_blocks * s->block_size >= ((int64_t)1 << 31))
        return PA_ERR_INVALID_ARG;
    if (N > s->num_rows) return PA_ERR_INVALID_ARG;  // the rows of a call are distinct
    if (!s->tables || !s->lens || !s->free_list || !s->free_count || !workspace) return PA_ERR_INVALID_ARG;
    if (((uintptr_t)workspace & 255) != 0) return PA_ERR_INVALID_ARG;
    if (workspace_bytes < tables_workspace(N, s->num_rows)) return PA_ERR_WORKSPACE;
    a->tables = s->tables;
    a->lens = s->lens;
    a->lens_out = s->lens_out ? s->lens_out : s->lens;
    a->free_list = s->free_list;
    a->free_count = s->free_count;
    a->free_count_out = s->free_count_out ? s->free_count_out : s->free_count;
    a->R = s->num_rows;
    a->W = s->max_blocks_per_row;
    a->NB = s->num_blocks;
    a->B = s->block_size;
    a->rows = rows;
    a->N = N;
    uint8_t *ws = (uint8_t *)workspace;
    a->ctl = (int32_t *)ws;
    a->reqs = (TableReq *)(ws + 256);
    a->claims = (int32_t *)(ws + 256 + align256(sizeof(TableReq) * (size_t)std::max(N, 1)));
    a->err = device_error_word();
    return a->err ? PA_OK : PA_ERR_CUDA;
}

pa_status_t launch_tables(const void *plan, const void *fill, dim3 grid, TablesArgs &a, cudaStream_t s) {
    cudaGetLastError();
    void *args[] = {&a};
    if (launch_pdl(plan, dim3(1), dim3(1024), args, 0, s) != cudaSuccess) return PA_ERR_CUDA;
    if (launch_pdl(fill, grid, dim3(256), args, 0, s) != cudaSuccess) return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_tables_workspace_bytes(int32_t num_reqs, int32_t num_rows) {
    return num_reqs < 0 || num_rows <= 0 ? 0 : tables_workspace(num_reqs, num_rows);
}

extern "C" pa_status_t pa_extend_tables(const pa_tables_t *state, const int32_t *rows, const int32_t *new_lens,
                                        int32_t num_reqs, int32_t *batch_tables, int32_t batch_width, int32_t *seq_lens,
                                        int32_t *cu_q_lens, int32_t *slot_mapping, int32_t max_tokens, void *workspace,
                                        size_t workspace_bytes, pa_stream_t stream) try {
    TablesArgs a{};
    const pa_status_t st = tables_args(state, rows, num_reqs, workspace, workspace_bytes, &a);
    if (st != PA_OK) return st;
    if (max_tokens < 0 || (batch_tables && batch_width <= 0)) return PA_ERR_INVALID_ARG;
    if (batch_tables && (int64_t)num_reqs * batch_width >= ((int64_t)1 << 31)) return PA_ERR_INVALID_ARG;
    if (!cu_q_lens || (max_tokens > 0 && !slot_mapping) || (num_reqs > 0 && (!new_lens || !seq_lens))) return PA_ERR_INVALID_ARG;
    a.new_lens = new_lens;
    a.batch_tables = num_reqs > 0 ? batch_tables : nullptr;
    a.BW = batch_width;
    a.seq_lens = seq_lens;
    a.cu_q = cu_q_lens;
    a.slots = slot_mapping;
    a.max_tokens = max_tokens;
    // slices of a request: 1024 table entries each
    const int64_t width = a.batch_tables ? a.BW : std::min<int64_t>(a.W, (int64_t)max_tokens / a.B + 2);
    const int64_t y = std::min<int64_t>((std::max<int64_t>(width, max_tokens / std::max(num_reqs, 1)) + 1023) / 1024, 64);
    return launch_tables((const void *)tables_plan_kernel<false>, (const void *)extend_fill_kernel,
                         dim3(std::max(num_reqs, 1), (unsigned)std::max<int64_t>(y, 1)), a, (cudaStream_t)stream);
} catch (...) {
    return host_failure();
}

extern "C" pa_status_t pa_release_tables(const pa_tables_t *state, const int32_t *rows, int32_t num_reqs, void *workspace,
                                         size_t workspace_bytes, pa_stream_t stream) try {
    TablesArgs a{};
    const pa_status_t st = tables_args(state, rows, num_reqs, workspace, workspace_bytes, &a);
    if (st != PA_OK) return st;
    const int64_t y = std::min<int64_t>(((int64_t)a.W + 1023) / 1024, 64);
    cudaStream_t s = (cudaStream_t)stream;
    if (num_reqs == 0) {  // the state's copies are still made
        cudaGetLastError();
        void *args[] = {&a};
        return launch_pdl((const void *)tables_plan_kernel<true>, dim3(1), dim3(1024), args, 0, s) == cudaSuccess &&
                       cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    }
    return launch_tables((const void *)tables_plan_kernel<true>, (const void *)release_fill_kernel,
                         dim3(num_reqs, (unsigned)y), a, s);
} catch (...) {
    return host_failure();
}
