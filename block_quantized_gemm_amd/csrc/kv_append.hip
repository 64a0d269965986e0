// kv_append.hip -- rows of keys and values into the pages of a cache.
//
// Keys are copied row by row; values go into blocks of 32 tokens x D channels,
// transposed.  A thread owns 8 consecutive positions (a 16-byte run of each of
// its channels) x 8 channels of one head's keys or values: eight 16-byte loads
// of row pieces, for values the 8 x 8 transpose in registers (one byte permute
// per output dword), eight 16-byte stores.  Four such threads side by side fill the 64 bytes of
// a channel, D / 8 of them take a whole row of the head, so loads and key
// stores move whole rows and value stores whole channels.
//
// A run that is only partly written (the ends of a prompt, the few tokens of
// an accepted path) keeps its other tokens: the thread reads the channel's 16
// bytes and writes them back merged.  No other thread of the call writes them,
// and a merged store costs one memory request per channel where single
// elements cost one per token and channel.
//
// Measured (8 heads of 128, one MI355X): two prompts of 8,190 rows into one
// layer 32 to 33 us (134 MB moved, 4.1 TB/s), bound by the bytes; 32 paths of 1
// to 8 rows into 16 layers 26 to 27.5 us (52 us with element stores), bound by
// the value blocks' lines, of which a few rows fill a part: 50 MB are read and
// 690,000 lines' parts written (a quarter of them 64 whole bytes) for rows of
// 10.7 MB; one path into 16 layers
// 4.9 us in the kernel, three dependent memory round trips (lengths and path,
// page, rows).  Keys and values in one thread took 43 us on the prompts: their
// 300 registers left one wave per SIMD.
#include "tree_internal.h"
#include "vq_device.h"

namespace vq {

namespace {

constexpr int kThreads = 256;
constexpr int kRun = 8;  // positions of a thread

struct KArgs {
    const uint16_t *k, *v;
    uint16_t *k_cache, *v_cache;
    const int32_t *page_table, *ctx_len, *path, *count;
    int32_t *len_out;
    int64_t k_stride, v_stride;
    int layers, batch, n, kv_heads, page_shift, n_pages, max_pages, blocks;
};

template <int D>
__global__ __launch_bounds__(kThreads, 4) void kv_append_kernel(KArgs a, int64_t items) {
    const bool keys = blockIdx.y == 1;
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int cap = a.max_pages << a.page_shift;
    if (a.len_out && !keys && item < a.batch) {
        const int ctx = min(max(a.ctx_len[item], 0), cap);
        const int cnt = a.count ? min(max(a.count[item], 0), a.n) : a.n;
        a.len_out[item] = min(ctx + cnt, cap);
    }
    if (item >= items)
        return;
    // channels fastest, then the runs of a block, heads, blocks, sequences, layers
    constexpr int kGroups = D / 8, kRuns = kVBlock / kRun;
    const int d = (int)(item % kGroups) * 8, run = (int)(item / kGroups % kRuns);
    int64_t rest = item / (kGroups * kRuns);
    const int h = (int)(rest % a.kv_heads);
    rest /= a.kv_heads;
    const int block = (int)(rest % a.blocks);
    rest /= a.blocks;
    const int b = (int)(rest % a.batch), layer = (int)(rest / a.batch);

    const int ctx = min(max(a.ctx_len[b], 0), cap);
    const int cnt = a.count ? min(max(a.count[b], 0), a.n) : a.n;
    const int pos = (ctx / kVBlock + block) * kVBlock + run * kRun;  // the run's first position
    const int end = min(ctx + cnt, cap);
    if (pos >= end || pos + kRun <= ctx)
        return;
    const int page = a.page_table[(int64_t)b * a.max_pages + (pos >> a.page_shift)];
    if (page < 0 || page >= a.n_pages)
        return;

    uint32_t valid = 0;  // bit t: position pos + t is written
    int64_t row[kRun];
#pragma unroll
    for (int t = 0; t < kRun; ++t) {
        const int i = pos + t - ctx;
        int from = -1;
        if (i >= 0 && pos + t < end)
            from = a.path ? a.path[(int64_t)b * a.n + i] : i;
        const bool ok = from >= 0 && from < a.n;
        valid |= (ok ? 1u : 0u) << t;
        row[t] = ((int64_t)layer * a.batch + b) * a.n + (ok ? from : 0);
    }
    const int off = pos & ((1 << a.page_shift) - 1);
    const int64_t head = ((((int64_t)layer * a.n_pages + page) * a.kv_heads + h) << a.page_shift) * D;
    const uint16_t *src = (keys ? a.k : a.v) + (int64_t)h * D + d;
    const int64_t stride = keys ? a.k_stride : a.v_stride;
    u32x4 x[kRun];
#pragma unroll
    for (int t = 0; t < kRun; ++t)
        x[t] = valid >> t & 1 ? ld16(src + row[t] * stride) : u32x4{0u, 0u, 0u, 0u};
    if (keys) {
        uint16_t *kd = a.k_cache + head + (int64_t)off * D + d;
#pragma unroll
        for (int t = 0; t < kRun; ++t)
            if (valid >> t & 1)
                *reinterpret_cast<u32x4 *>(kd + (int64_t)t * D) = x[t];
        return;
    }
    uint16_t *vd = a.v_cache + head + (int64_t)(off / kVBlock * kVBlock) * D + d * kVBlock + off % kVBlock;
    u32x4 old[8];
    if (valid != 0xFFu)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            old[e] = ld16(vd + e * kVBlock);
    if (valid == 0)
        return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        u32x4 out;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const uint32_t lo = x[2 * y][e >> 1], hi = x[2 * y + 1][e >> 1];  // tokens 2 y and 2 y + 1
            out[y] = __builtin_amdgcn_perm(hi, lo, e & 1 ? 0x07060302u : 0x05040100u);
        }
        if (valid != 0xFFu)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint32_t mine =
                    (valid >> (2 * y) & 1 ? 0xFFFFu : 0u) | (valid >> (2 * y + 1) & 1 ? 0xFFFF0000u : 0u);
                out[y] = (out[y] & mine) | (old[e][y] & ~mine);
            }
        *reinterpret_cast<u32x4 *>(vd + e * kVBlock) = out;
    }
}

// Blocks of 32 positions that n rows can touch wherever they begin.
int64_t blocks_of(int64_t n) { return (n + kVBlock - 2) / kVBlock + 1; }

// Threads of each half of the grid (values, keys).
int64_t items_of(int64_t n_layers, int64_t batch, int64_t n, int64_t kv_heads, int64_t head_dim) {
    return n_layers * batch * blocks_of(n) * kv_heads * (kVBlock / kRun) * (head_dim / 8);
}
int64_t groups_of(int64_t items, int64_t batch) { return (std::max(items, batch) + kThreads - 1) / kThreads; }

}  // namespace

bool kv_append_fits(int64_t n_layers, int64_t batch, int64_t n, int64_t kv_heads, int64_t head_dim) {
    return groups_of(items_of(n_layers, batch, n, kv_heads, head_dim), batch) * kThreads <= 0xFFFFFFFFll;
}

hipError_t launch_kv_append(const KvAppendArgs &p) {
    KArgs a{static_cast<const uint16_t *>(p.k), static_cast<const uint16_t *>(p.v),
            static_cast<uint16_t *>(p.k_cache), static_cast<uint16_t *>(p.v_cache), p.page_table, p.ctx_len, p.path,
            p.count, p.len_out, p.k_stride, p.v_stride, p.n_layers, p.batch, p.n, p.kv_heads,
            __builtin_ctz((unsigned)p.page_size), p.n_pages, p.max_pages, 0};
    a.blocks = (int)blocks_of(p.n);
    const int64_t items = items_of(p.n_layers, p.batch, p.n, p.kv_heads, p.head_dim);
    const int64_t groups = groups_of(items, p.batch);
    const dim3 grid((unsigned)groups, 2), threads(kThreads);  // values, then keys
    if (p.head_dim == 64)
        hipLaunchKernelGGL(kv_append_kernel<64>, grid, threads, 0, p.stream, a, items);
    else if (p.head_dim == 128)
        hipLaunchKernelGGL(kv_append_kernel<128>, grid, threads, 0, p.stream, a, items);
    else
        hipLaunchKernelGGL(kv_append_kernel<256>, grid, threads, 0, p.stream, a, items);
    return hipGetLastError();
}

}  // namespace vq
