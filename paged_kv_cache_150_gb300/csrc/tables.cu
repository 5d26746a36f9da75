// A step's tables on the GPU (pa_extend_tables, pa_release_tables): blocks for
// the new tokens of a batch of requests taken off a free stack, its block
// tables, lengths, row offsets and slot map; and blocks given back.
//
// With L_i tokens before the step and n_i new ones, block size B:
//   request i takes ceil((L_i + n_i) / B) - ceil(L_i / B) blocks, whose place on
//   the stack is an exclusive prefix sum over the requests; token t of it has the
//   slot table[p / B] * B + p % B, p = L_i + t.
// One CTA checks every request and scans (a call that cannot be met changes
// nothing, so nothing is written before the last check); small batches are
// filled in by the same CTA, larger ones by a second kernel of (request, slice)
// CTAs.  Slots of new blocks are read off the stack, not off the table entries
// that the same kernel writes, so nothing waits for them.  Everything is int32
// and a call moves some bytes per request beside the table rows: it is bound by
// the latency of its launches and of three dependent reads (row, length, block)
// until the tables reach megabytes.  One request given back and four extended,
// tables of 8 blocks: 7.3 us for the two calls; 64 given back and 1024 extended by
// 1 to 512 tokens, tables of 2048 blocks (13.4 MB): 14.4 us.
#include "prefill_plan.cuh"  // last_at_most

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
    int32_t *claims;  // [R] the first request that names each row
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

// What a call wants of one request, and why it cannot have it.
struct TableLook {
    int32_t row, old, len, blocks;  // blocks taken or given back
    unsigned int bad;
};
// claims: of the requests that name one row the first is the row's, the others refuse the call.
template <bool kRelease>
__device__ __forceinline__ TableLook look_at(const TablesArgs &a, int32_t i, int32_t row, int32_t claim) {
    TableLook q{row, 0, 0, 0, 0u};
    const int64_t max_len = (int64_t)a.W * a.B;
    if (row < 0 || claim != i) {
        q.bad = kErrBounds;
        q.row = -1;
        return q;
    }
    const int32_t old = a.lens[row], n = kRelease ? 0 : a.new_lens[i];
    if (old < 0 || old > max_len) {
        q.bad = kErrLength;
        return q;
    }
    q.old = q.len = old;
    if (kRelease) {
        q.blocks = blocks_of(old, a.B);
        return q;
    }
    if (n < 0 || (int64_t)old + n > max_len) {
        q.bad = kErrLength;
        return q;
    }
    q.len = old + n;
    const int32_t nb = blocks_of(q.len, a.B);
    q.blocks = nb - blocks_of(old, a.B);
    if (a.batch_tables && nb > a.BW) q.bad = kErrBounds;
    return q;
}

// Inclusive scans of blocks and tokens over 1024 threads (the tokens' sum may
// pass 32 bits), the totals, and all threads' bad bits together.
struct TableScan {
    int32_t blocks[32];
    int64_t tokens[32];
    unsigned int bad[32];
};
__device__ __forceinline__ void scan_1024(TableScan *s, int32_t &blocks, int64_t &tokens, unsigned int &bad,
                                          int32_t *all_blocks, int64_t *all_tokens) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t b = __shfl_up_sync(0xffffffffu, blocks, o);
        const int64_t t = __shfl_up_sync(0xffffffffu, tokens, o);
        if (lane >= o) blocks += b, tokens += t;
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    __syncthreads();  // the previous scan's reads
    if (lane == 31) s->blocks[w] = blocks, s->tokens[w] = tokens, s->bad[w] = bad;
    __syncthreads();
    int32_t wb = s->blocks[lane];  // every warp scans the warps' sums
    int64_t wt = s->tokens[lane];
    bad = __reduce_or_sync(0xffffffffu, s->bad[lane]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t b = __shfl_up_sync(0xffffffffu, wb, o);
        const int64_t t = __shfl_up_sync(0xffffffffu, wt, o);
        if (lane >= o) wb += b, wt += t;
    }
    *all_blocks = __shfl_sync(0xffffffffu, wb, 31);
    *all_tokens = __shfl_sync(0xffffffffu, wt, 31);
    const int before = w > 0 ? w - 1 : 0;
    wb = __shfl_sync(0xffffffffu, wb, before), wt = __shfl_sync(0xffffffffu, wt, before);
    if (w > 0) blocks += wb, tokens += wt;
}

// A block of a request's table: its own, or a new one off the stack.
__device__ __forceinline__ int32_t block_at(const TablesArgs &a, const int32_t *row, int32_t j, int32_t nb0, int32_t top) {
    return j < nb0 ? row[j] : a.free_list[top - (j - nb0)];
}
__device__ __forceinline__ int32_t slot_in(const TablesArgs &a, int32_t block, int32_t off) {
    const bool good = block >= 0 && block < a.NB;
    if (!good) atomicOr(a.err, kErrBounds);
    return good ? block * a.B + off : -1;
}

constexpr int32_t kClaimsSmem = 4096;  // rows whose claims are kept in shared memory
// Table entries and slots (or blocks given back) of a call that one CTA fills in
// as well: 4096 more take it about 1 us, the second kernel's launch 2.
constexpr int64_t kOneCta = 8192;

// Checks and prefix sums of a call, and its filling in where it is small
// (kFill).  kRelease: the requests give back all their blocks; else they take
// blocks for their new tokens.
template <bool kRelease, bool kFill>
__global__ void __launch_bounds__(1024) tables_plan_kernel(const __grid_constant__ TablesArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ TableScan scan;
    __shared__ int32_t claims_s[kClaimsSmem];
    __shared__ TableReq reqs_s[kFill ? 1024 : 1];
    __shared__ int32_t cu_s[kFill ? 1025 : 1];
    const int tid = threadIdx.x;
    const int32_t count = *a.free_count;
    int32_t *claims = a.R <= kClaimsSmem ? claims_s : a.claims;
    int32_t row0 = -1;  // row of this thread's first request
    for (int32_t i = tid; i < a.N; i += 1024) {
        const int32_t row = row_of(a, i);
        if (i == tid) row0 = row;
        if (row >= 0) claims[row] = i;
    }
    __syncthreads();
    auto look = [&](int32_t i) {
        const int32_t row = i == tid ? row0 : row_of(a, i);
        return look_at<kRelease>(a, i, row, row >= 0 ? claims[row] : -1);
    };
    // One pass over the requests settles whether the call is met, another (the
    // same one for up to 1024 requests) writes what it gives.
    unsigned int bad = count < 0 || count > a.NB ? kErrBounds : 0u;
    int32_t at = 0, all_blocks = 0;
    int64_t cu = 0, all_tokens = 0;
    TableLook mine{-1, 0, 0, 0, 0u};
    int32_t blocks = 0;
    int64_t tokens = 0;
    for (int32_t base = 0; base < a.N || base == 0; base += 1024) {
        const int32_t i = base + tid;
        mine = TableLook{-1, 0, 0, 0, 0u};
        if (i < a.N) mine = look(i);
        blocks = mine.blocks;
        tokens = mine.len - mine.old;
        bad |= mine.bad;
        int32_t b;
        int64_t t;
        scan_1024(&scan, blocks, tokens, bad, &b, &t);
        all_blocks += b;  // N rows of at most 2^31 entries in all
        all_tokens += t;
    }
    if (bad) {
        // A row named twice stays the first request's, whichever store came last
        // (here, where the call is refused already: 0.4 us in front of every scan).
        for (int32_t i = tid; i < a.N; i += 1024) {
            const int32_t row = i == tid ? row0 : row_of(a, i);
            if (row >= 0 && *(volatile int32_t *)(claims + row) != i) atomicMin(claims + row, i);
        }
        __syncthreads();
        if (tid < a.N && a.N <= 1024) mine = look(tid);
    }
    if (kRelease) {
        if (!bad && (int64_t)count + all_blocks > a.NB) bad = kErrBounds;  // more blocks than the pool has
    } else if (!bad) {
        if (all_tokens > a.max_tokens)
            bad = kErrBounds;
        else if (all_blocks > count)
            bad = kErrNoBlocks;
    }
    const bool ok = bad == 0;
    for (int32_t base = 0; base < a.N; base += 1024) {
        const int32_t i = base + tid;
        if (a.N > 1024) {  // worked out again
            mine = TableLook{-1, 0, 0, 0, 0u};
            if (i < a.N) mine = look(i);
            blocks = mine.blocks;
            tokens = mine.len - mine.old;
            unsigned int none = 0;
            int32_t b;
            int64_t t;
            scan_1024(&scan, blocks, tokens, none, &b, &t);
            blocks += at, tokens += cu;
            at += b, cu += t;
        }
        if (i < a.N) {
            const int32_t n = mine.len - mine.old;
            TableReq q{mine.row, mine.old, ok ? mine.len : mine.old, ok ? blocks - mine.blocks : 0};
            if (kRelease && !ok) q.row = -1;
            if (kFill)
                reqs_s[i] = q;
            else
                a.reqs[i] = q;
            if (!kRelease) {
                const int32_t c = ok ? (int32_t)tokens - n : 0;
                a.cu_q[i] = c;
                if (kFill) cu_s[i] = c;
                a.seq_lens[i] = q.len;
            }
        }
    }
    const int32_t total = ok ? (int32_t)all_tokens : 0;  // new tokens
    if (tid == 0) {
        if (!kRelease) {
            a.cu_q[a.N] = total;
            if (kFill) cu_s[a.N] = total;
        }
        a.ctl[0] = count;
        *a.free_count_out = !ok ? count : kRelease ? count + all_blocks : count - all_blocks;
        if (!ok) atomicOr(a.err, bad);
    }
    __syncthreads();  // the last reads of lens, which lens_out may be; the lists in shared memory
    if (a.lens_out != a.lens) {
        for (int32_t r = tid; r < a.R; r += 1024) a.lens_out[r] = a.lens[r];
        __syncthreads();
    }
    if (ok) {
        if (a.N <= 1024) {
            if (tid < a.N) a.lens_out[mine.row] = kRelease ? 0 : mine.len;
        } else {
            for (int32_t i = tid; i < a.N; i += 1024) {
                const TableReq q = a.reqs[i];  // this thread's own
                a.lens_out[q.row] = kRelease ? 0 : q.len;
            }
        }
    }
    if constexpr (kFill) {
        if (kRelease) {
            // the stack's new entries, by the request that they come from
            for (int32_t e = tid; ok && e < all_blocks; e += 1024) {
                int32_t lo = 0, hi = a.N - 1;
                while (lo < hi) {
                    const int32_t mid = (lo + hi + 1) >> 1;
                    if (reqs_s[mid].first <= e)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                const TableReq q = reqs_s[lo];
                const int32_t b = a.tables[(int64_t)q.row * a.W + (e - q.first)];
                if (b < 0 || b >= a.NB) atomicOr(a.err, kErrBounds);
                a.free_list[count + e] = b;
            }
        } else {
            const int32_t width = a.batch_tables ? a.BW : a.W;
            const uint32_t entries = (uint32_t)a.N * (uint32_t)width;  // at most kOneCta
            for (uint32_t e = tid; e < entries; e += 1024) {
                const uint32_t i = e / (uint32_t)width;
                const int32_t j = (int32_t)(e - i * (uint32_t)width);
                const TableReq q = reqs_s[i];
                const int32_t nb0 = blocks_of(q.old, a.B), nb1 = blocks_of(q.len, a.B);
                int32_t *row = a.tables + (int64_t)max(q.row, 0) * a.W;
                int32_t b = -1;
                if (q.row >= 0 && j < nb1) {
                    b = block_at(a, row, j, nb0, count - 1 - q.first);
                    if (j >= nb0) row[j] = b;
                }
                if (a.batch_tables) a.batch_tables[e] = b;
            }
            for (int32_t t = tid; t < a.max_tokens; t += 1024) {
                int32_t slot = -1;
                if (t < total) {
                    const int32_t i = last_at_most(cu_s, a.N, t);
                    const TableReq q = reqs_s[i];
                    const int32_t p = q.old + (t - cu_s[i]), j = p / a.B;
                    slot = slot_in(a, block_at(a, a.tables + (int64_t)q.row * a.W, j, blocks_of(q.old, a.B), count - 1 - q.first),
                                   p - j * a.B);
                }
                a.slots[t] = slot;
            }
        }
    }
}

// Tables and slots: CTA (i, y) takes the y-th part of request i's.  kVec: rows
// and batch rows of whole, aligned 16-byte vectors.
template <bool kVec>
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
    const int32_t nb0 = q.row < 0 ? 0 : blocks_of(q.old, a.B), nb1 = q.row < 0 ? 0 : blocks_of(q.len, a.B);
    int32_t *row = a.tables + (int64_t)max(q.row, 0) * a.W;
    if (a.batch_tables) {
        int32_t *out = a.batch_tables + (int64_t)i * a.BW;
        constexpr int E = kVec ? 4 : 1;
        for (int32_t j = tid * E; j < a.BW; j += stride * E) {
            if (kVec && (j + 4 <= nb0 || j >= nb1)) {  // blocks that it had, or none
                const int4 none = make_int4(-1, -1, -1, -1);
                *reinterpret_cast<int4 *>(out + j) = j >= nb1 ? none : *reinterpret_cast<const int4 *>(row + j);
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    int32_t b = -1;
                    if (j + k < nb1) {
                        b = block_at(a, row, j + k, nb0, top);
                        if (j + k >= nb0) row[j + k] = b;
                    }
                    out[j + k] = b;
                }
            }
        }
    } else {
        for (int32_t j = nb0 + tid; j < nb1; j += stride) row[j] = a.free_list[top - (j - nb0)];
    }
    for (int32_t t = tid; t < q.len - q.old; t += stride) {
        const int32_t p = q.old + t, j = p / a.B;
        a.slots[cu + t] = slot_in(a, block_at(a, row, j, nb0, top), p - j * a.B);
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

constexpr int32_t kMostEntries = 1 << 30;  // of a loop: its index and a stride stay within 32 bits

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
    if (s->num_rows > kMostEntries || s->max_blocks_per_row > kMostEntries) return PA_ERR_UNSUPPORTED;
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
    return PA_OK;
}

pa_status_t launch_tables(const void *plan, const void *fill, dim3 grid, TablesArgs &a, cudaStream_t s) {
    a.err = device_error_word();
    if (!a.err) return PA_ERR_CUDA;
    cudaGetLastError();
    void *args[] = {&a};
    if (launch_pdl(plan, dim3(1), dim3(1024), args, 0, s) != cudaSuccess) return PA_ERR_CUDA;
    if (fill && launch_pdl(fill, grid, dim3(256), args, 0, s) != cudaSuccess) return PA_ERR_CUDA;
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
    if (max_tokens > kMostEntries || (batch_tables && batch_width > kMostEntries)) return PA_ERR_UNSUPPORTED;
    if (!cu_q_lens || (max_tokens > 0 && !slot_mapping) || (num_reqs > 0 && (!new_lens || !seq_lens))) return PA_ERR_INVALID_ARG;
    a.new_lens = new_lens;
    a.batch_tables = num_reqs > 0 ? batch_tables : nullptr;
    a.BW = batch_width;
    a.seq_lens = seq_lens;
    a.cu_q = cu_q_lens;
    a.slots = slot_mapping;
    a.max_tokens = max_tokens;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t width = a.batch_tables ? a.BW : a.W;
    if (num_reqs <= 1024 && num_reqs * width + max_tokens <= kOneCta)
        return launch_tables((const void *)tables_plan_kernel<false, true>, nullptr, dim3(1), a, s);
    // slices of a request: 1024 table entries each, or its share of the tokens
    const int64_t most = std::max<int64_t>(a.batch_tables ? a.BW : std::min<int64_t>(a.W, (int64_t)max_tokens / a.B + 2),
                                           max_tokens / std::max(num_reqs, 1));
    const unsigned y = (unsigned)std::max<int64_t>(std::min<int64_t>((most + 1023) / 1024, 64), 1);
    const bool vec = a.batch_tables && a.W % 4 == 0 && a.BW % 4 == 0 && (((uintptr_t)a.tables | (uintptr_t)a.batch_tables) & 15) == 0;
    return launch_tables((const void *)tables_plan_kernel<false, false>,
                         vec ? (const void *)extend_fill_kernel<true> : (const void *)extend_fill_kernel<false>,
                         dim3(std::max(num_reqs, 1), y), a, s);
} catch (...) {
    return host_failure();
}

extern "C" pa_status_t pa_release_tables(const pa_tables_t *state, const int32_t *rows, int32_t num_reqs, void *workspace,
                                         size_t workspace_bytes, pa_stream_t stream) try {
    TablesArgs a{};
    const pa_status_t st = tables_args(state, rows, num_reqs, workspace, workspace_bytes, &a);
    if (st != PA_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    if (num_reqs <= 1024 && (int64_t)num_reqs * a.W <= kOneCta)
        return launch_tables((const void *)tables_plan_kernel<true, true>, nullptr, dim3(1), a, s);
    const unsigned y = (unsigned)std::min<int64_t>(((int64_t)a.W + 1023) / 1024, 64);
    return launch_tables((const void *)tables_plan_kernel<true, false>, (const void *)release_fill_kernel,
                         dim3(num_reqs, y), a, s);
} catch (...) {
    return host_failure();
}
