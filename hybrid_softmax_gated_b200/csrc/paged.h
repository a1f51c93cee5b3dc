// Paged KV cache: what the host entries (paged.cu) hand to the kernels.
#pragma once

#include "internal.h"

namespace arl2 {

// Bits of the paged handle's error word.
enum : int {
    kErrPagedTimeout = 1 << 0,  // a bounded wait ran out
    kErrPagedTable = 1 << 1,    // offsets, lengths or a page number out of range
};

constexpr int kPagedMaxSeqs = 1024;

// Heads and pages of a pool: [pages][Hk][page][d].
struct PagedGeom {
    int Hq, Hk, G;        // G = Hq / Hk query heads read one key head
    int d;
    int pages, page_log2; // page = 1 << page_log2 tokens
};

struct PagedPool {
    void* k;
    void* v;
    float* ks;            // [pages][Hk][page], e4m3 only
    float* vs;
};

// The batch's device tables (see include/arl2.h).
struct PagedSeqs {
    int S, tokens, max_pages;
    const int* q_off;
    const int* kv_len;
    const int* table;
};

// Query at position p: keys j < min(total, E) with E = (p / block + 1) block,
// and (window) j >= E - window or j < sinks; window and sinks in tokens,
// window = 0: none.
struct PagedMask {
    int block, window, sinks;
};

// Partial results of query tiles that several CTAs share, and the counters
// of their arrivals (zero between launches).
struct PagedWork {
    float* o;             // [piece][rows][d]
    float2* ml;           // [piece][rows]: running max (log2 units), row sum
    int* arrived;         // [CTA]
};
// Rows of partials the workspace holds per SM: two pieces per CTA, and a
// kernel's CTAs per SM times its tile rows stay within this.
constexpr int kPagedRowsPerSm = 512;

struct PagedAttend {
    PagedGeom g;
    PagedPool pool;
    PagedSeqs seqs;
    PagedMask mask;
    PagedWork work;
    const void* q;
    long long q_stride;
    void* out;
    float scale;
    int* err;
};

cudaError_t launch_paged_write(bool bf16, bool e4m3, const PagedGeom& g, const PagedPool& pool, const PagedSeqs& seqs,
                               const void* k, long long k_stride, const void* v, long long v_stride, int* err,
                               cudaStream_t st);
cudaError_t launch_paged_read(bool bf16, bool e4m3, const PagedGeom& g, const PagedPool& pool, const PagedSeqs& seqs,
                              const int* starts, void* k, void* v, int* err, cudaStream_t st);

// fp32 arithmetic, any head width up to 128 (paged_simt.cu).
cudaError_t paged_simt_init();
cudaError_t launch_paged_simt(bool bf16, bool e4m3, const PagedAttend& a, int max_new, int max_ctas,
                              cudaStream_t st);

// bf16 tensors, head width 128, on the tensor cores (paged_tc.cu).
bool paged_tc_init();
cudaError_t launch_paged_tc(bool e4m3, const PagedAttend& a, int max_ctas, cudaStream_t st);
// The same for tiles of `rows` <= 16 query rows (paged_few.cu).
bool paged_few_init();
cudaError_t launch_paged_few(bool e4m3, const PagedAttend& a, int rows, int max_ctas, cudaStream_t st);

}  // namespace arl2
