// api_diff.cu -- the C ABI of rotary positions and of differential attention: argument checks,
// tensor maps and launches.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "api_internal.h"
#include "diff_params.h"

using namespace gb300;

// ------------------------------------------------------------------ rotary positions
extern "C" attn_status_t attn_rope_bf16(const void* q, const void* k, void* q_out, void* k_out,
                                        const int* positions, const float* inv_freq, const int* axis,
                                        const long long* strides, int B, int N, int Hq, int Hk, int d, int rot,
                                        int axes, int interleaved, int inverse, void* stream)
{
    if (B < 0 || N < 0 || Hq < 1 || Hk < 0 || axes < 1 || !strides) return ATTN_ERR_INVALID_ARG;
    if (d < 16 || d > 256 || d % 16 != 0 || rot < 16 || rot > d || rot % 16 != 0) return ATTN_ERR_UNSUPPORTED;
    if ((long long)B * N > 0x7fffffffLL || Hq > 65535 || Hk > 65535 || axes > 255) return ATTN_ERR_UNSUPPORTED;
    // the threads of the longest launch (rope.cu), eight heads each, stay in 32 bits
    const int heads = Hq + Hk, each = heads < 8 ? heads : 8;
    if (((long long)B * N * ((heads + each - 1) / each) * (d / 16)) > 0xffffff00LL) return ATTN_ERR_UNSUPPORTED;
    if (B == 0 || N == 0) return ATTN_OK;
    if (!q || !q_out || !positions || !inv_freq || (Hk > 0 && (!k || !k_out))) return ATTN_ERR_INVALID_ARG;
    const int tensors = Hk > 0 ? 4 : 2;      // q, q_out, k, k_out
    const void* at[4] = {q, q_out, k, k_out};
    for (int i = 0; i < tensors; ++i) {
        if (!aligned(at[i], 16)) return ATTN_ERR_MISALIGNED;
        for (int s = 0; s < 3; ++s)
            if (strides[3 * i + s] % 8 != 0) return ATTN_ERR_MISALIGNED;
    }
    if (!aligned(positions, 4) || !aligned(inv_freq, 4) || !aligned(axis, 4)) return ATTN_ERR_MISALIGNED;
    DeviceInfo* dev = nullptr;
    const attn_status_t st = device_info(&dev);
    if (st != ATTN_OK) return st;
    RopeParams p;
    std::memset(&p, 0, sizeof(p));
    p.q = {q, q_out, strides[0], strides[1], strides[2], strides[3], strides[4], strides[5]};
    if (Hk > 0) p.k = {k, k_out, strides[6], strides[7], strides[8], strides[9], strides[10], strides[11]};
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.axis = axis;
    p.tokens = B * N;
    p.N = N;
    p.Hq = Hq;
    p.Hk = Hk;
    p.d = d;
    p.rot = rot;
    p.axes = axes;
    p.interleaved = interleaved ? 1 : 0;
    p.inverse = inverse ? 1 : 0;
    return launch_rope(p, dev->sm_count, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// ------------------------------------------------------------------ differential attention
namespace {

constexpr int kDiffMaxRows = 0x7fffff00;   // a last tile's rows stay in int

// What every entry point below checks of its sizes.
attn_status_t diff_sizes(int H, int Hkv, int d, float scale)
{
    if (H < 1 || Hkv < 1 || H % Hkv != 0) return ATTN_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// Maps over q [.., 2H, .., d], k [.., 2Hkv, .., d] and v or o [.., heads, .., 2d], batched (T < 0: [B, heads, N,
// width]) or packed [T, heads, width].
bool diff_map(CUtensorMap* m, const void* base, int width, int heads, int B, int N, int T, int box_rows)
{
    if (T < 0)
        return encode_rows(m, base, width, N, width, (long long)B * heads, (long long)N * width, box_rows);
    return encode_rows(m, base, width, T, (long long)heads * width, heads, width, box_rows);
}

struct DiffShape {
    int B, H, Hkv, N, d;          // packed: N the longest sequence
    const int* cu_seqlens;        // packed layout, else null
    int num_seqs, T;              // T < 0: batched
    float scale;
    int causal, window;
};

attn_status_t diff_fwd(const void* q, const void* k, const void* v, const float* lam, void* o, float* lse, void* o2,
                       const DiffShape& s, void* stream, unsigned long long timeout_ns, int withhold)
{
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(o2, 16) ||
        !aligned(lam, 4) || !aligned(lse, 4) || !aligned(s.cu_seqlens, 4))
        return ATTN_ERR_MISALIGNED;
    if (s.N > kDiffMaxRows || s.T > kDiffMaxRows || s.H > 65535) return ATTN_ERR_UNSUPPORTED;
    const bool packed = s.T >= 0;
    const int parts = s.d / 64;
    const long long heads = (packed ? (long long)s.num_seqs : (long long)s.B) * s.H * parts;
    const long long blocks = ((long long)s.N + 127) / 128, pairs = heads * ((blocks + 1) / 2);
    DeviceInfo* dev = nullptr;
    const attn_status_t st = device_info(&dev);
    if (st != ATTN_OK) return st;
    // sub-unit indices, and a walk's step past the last one, stay in int; so do head coordinates
    if (2 * pairs + 4LL * dev->sm_count > 0x7fffffffLL || 2 * heads > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
    alignas(64) DiffFwdMaps m;
    if (!diff_map(&m.q, q, s.d, 2 * s.H, s.B, s.N, s.T, 128) ||
        !diff_map(&m.k, k, s.d, 2 * s.Hkv, s.B, s.N, s.T, 128) ||
        !diff_map(&m.v, v, 2 * s.d, s.Hkv, s.B, s.N, s.T, 128) ||
        !diff_map(&m.k64, k, s.d, 2 * s.Hkv, s.B, s.N, s.T, 64) ||
        !diff_map(&m.v64, v, 2 * s.d, s.Hkv, s.B, s.N, s.T, 64))
        return ATTN_ERR_CUDA;
    DiffFwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.f.o = o;
    p.f.lse = lse;
    p.f.status = dev->status;
    p.f.BH = (int)heads;
    p.f.N = s.N;
    p.f.num_qblk = (int)blocks;
    p.f.num_units = (int)pairs;
    p.f.causal = s.causal ? 1 : 0;
    p.f.window = s.window > 0 && s.window < s.N ? s.window : 0;   // a wider one masks nothing
    p.f.c_log2 = (float)((double)s.scale * 1.4426950408889634);
    p.f.timeout_ns = timeout_ns;
    p.f.withhold_kv = withhold;
    p.f.cu_seqlens = s.cu_seqlens;
    p.f.num_seqs = s.num_seqs;
    p.f.H = s.H * parts;
    p.f.T = s.T;
    p.o2 = o2;
    p.lam = lam;
    p.H = s.H;
    p.Hkv = s.Hkv;
    // d = 128 without O_2: two launches of 12 d products in place of one of 16 d (diff_fwd_wide.cu), where the one would
    // take at least 25 steps of 128 x 128 scores an SM and there are units for every pair of SMs, half of them again.
    // Measured, one against two, 16 heads over 4: causal 1536 tokens (16 steps) 41 us against 45, 2048 (29) 62
    // against 54, 4096 198 against 159; 64 x 768 (18) 53 against 59, 64 x 1024 (30) 78 against 71; 4 heads, 4096 tokens
    // (64 units) 54 against 84; non-causal 64 x 512 (13) 39 against 35, 64 x 768 (30) 75 against 71.  So the few short calls without a mask that two
    // launches would serve better are given up, and so are packed ones whose lengths' mean is short beside their longest.
    cudaError_t e;
    const long long mean = packed ? s.T / s.num_seqs : s.N, seqs = packed ? s.num_seqs : s.B;
    long long keys = s.causal ? mean / 2 + 64 : mean;     // that a row sees, with what its tiles mask
    if (p.f.window > 0) keys = std::min(keys, (s.causal ? 1LL : 2LL) * p.f.window + 128);
    const long long steps = heads * ((mean + 127) / 128) * ((keys + 127) / 128);
    if (s.d == 128 && !o2 && mean > 256 && steps >= 25LL * dev->sm_count &&
        4 * seqs * s.H * ((mean + 255) / 256) >= 3LL * dev->sm_count) {
        auto shape = [&](int heads_of) {              // heads of one sequence
            DiffFwdParams r = p;
            r.f.H = heads_of;
            r.f.BH = (packed ? s.num_seqs : s.B) * heads_of;
            r.f.num_qblk = (int)(((long long)s.N + 255) / 256);
            r.f.num_units = r.f.BH * ((r.f.num_qblk + 1) / 2);
            return r;
        };
        e = launch_diff_fwd_wide(m, shape(2 * s.H), shape(s.H), dev->sm_count, static_cast<cudaStream_t>(stream));
    } else {
        e = launch_diff_fwd(m, p, s.d, dev->sm_count, static_cast<cudaStream_t>(stream));
    }
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// The workspace: three counters in 16 bytes, the table of packed sequences, then D_1 and D_2 of every row,
// laid out as the LSE.
constexpr size_t kDiffBwdHead = 2048;
static_assert(16 + sizeof(SortTab) <= kDiffBwdHead, "workspace");

attn_status_t diff_bwd(const void* q, const void* k, const void* v, const float* lam, const void* o, const void* o2,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv, float* dlam, void* workspace,
                       const DiffShape& s, void* stream, unsigned long long timeout_ns, int withhold)
{
    for (const void* t : {q, k, v, o, o2, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                          static_cast<const void*>(dv), static_cast<const void*>(workspace)})
        if (!aligned(t, 16)) return ATTN_ERR_MISALIGNED;
    if (!aligned(lam, 4) || !aligned(lse, 4) || !aligned(dlam, 4) || !aligned(s.cu_seqlens, 4))
        return ATTN_ERR_MISALIGNED;
    if (s.N > kDiffMaxRows || s.T > kDiffMaxRows || s.H > 65535) return ATTN_ERR_UNSUPPORTED;
    const bool packed = s.T >= 0;
    const int seqs = packed ? s.num_seqs : s.B;
    const long long tiles = ((long long)s.N + 127) / 128, units = tiles * seqs * 2 * s.H;
    DeviceInfo* dev = nullptr;
    const attn_status_t st = device_info(&dev);
    if (st != ATTN_OK) return st;
    // unit numbers, the counter's last value and the rows of the first kernel's grid stay in int
    const long long rows = (packed ? (long long)s.T : (long long)s.B * s.N) * s.H;
    if (units + 4LL * dev->sm_count > 0x7fffffffLL || rows / 8 > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
    alignas(64) DiffBwdMaps m;
    if (!diff_map(&m.q, q, s.d, 2 * s.H, s.B, s.N, s.T, 128) || !diff_map(&m.q64, q, s.d, 2 * s.H, s.B, s.N, s.T, 64) ||
        !diff_map(&m.dout, dout, 2 * s.d, s.H, s.B, s.N, s.T, 128) ||
        !diff_map(&m.dout64, dout, 2 * s.d, s.H, s.B, s.N, s.T, 64) ||
        !diff_map(&m.k, k, s.d, 2 * s.Hkv, s.B, s.N, s.T, 128) || !diff_map(&m.v, v, 2 * s.d, s.Hkv, s.B, s.N, s.T, 128))
        return ATTN_ERR_CUDA;
    DiffBwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.o = o;
    p.o2 = o2;
    p.dout = dout;
    p.lse = lse;
    p.lam = lam;
    p.next = static_cast<int*>(workspace);
    if (packed && seqs <= kSortMaxSeqs) p.tab = reinterpret_cast<SortTab*>(static_cast<uint8_t*>(workspace) + 16);
    p.delta = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kDiffBwdHead);
    p.dlam = dlam;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.status = dev->status;
    p.B = seqs;
    p.H = s.H;
    p.Hkv = s.Hkv;
    p.N = s.N;
    p.nt = (int)tiles;
    p.causal = s.causal ? 1 : 0;
    p.window = s.window > 0 && s.window < s.N ? s.window : 0;
    p.c_log2 = (float)((double)s.scale * 1.4426950408889634);
    p.scale = s.scale;
    p.timeout_ns = timeout_ns;
    p.withhold = withhold;
    p.cu_seqlens = s.cu_seqlens;
    p.T = s.T;
    return launch_diff_bwd(m, p, s.d, dev->sm_count, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK
                                                                                                       : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" attn_status_t attn_diff_fwd_bf16(const void* q, const void* k, const void* v, const float* lam, void* o,
                                            float* lse, void* o2, int B, int H, int Hkv, int N, int d, float scale,
                                            int causal, int window, void* stream)
{
    if (B < 1 || N < 1) return ATTN_ERR_INVALID_ARG;
    const attn_status_t st = diff_sizes(H, Hkv, d, scale);
    if (st != ATTN_OK) return st;
    if (!q || !k || !v || !lam || !o || !lse) return ATTN_ERR_INVALID_ARG;
    return diff_fwd(q, k, v, lam, o, lse, o2, {B, H, Hkv, N, d, nullptr, 0, -1, scale, causal, window}, stream,
                    kWaitTimeoutNs, 0);
}

extern "C" attn_status_t attn_diff_fwd_bf16_varlen(const void* q, const void* k, const void* v, const float* lam,
                                                   void* o, float* lse, void* o2, const int* cu_seqlens, int num_seqs,
                                                   int max_seqlen, int total_tokens, int H, int Hkv, int d,
                                                   float scale, int causal, int window, void* stream)
{
    if (num_seqs < 1 || total_tokens < 0 || max_seqlen < 0 || max_seqlen > total_tokens) return ATTN_ERR_INVALID_ARG;
    const attn_status_t st = diff_sizes(H, Hkv, d, scale);
    if (st != ATTN_OK) return st;
    if (total_tokens == 0 || max_seqlen == 0) return ATTN_OK;
    if (!q || !k || !v || !lam || !o || !lse || !cu_seqlens) return ATTN_ERR_INVALID_ARG;
    return diff_fwd(q, k, v, lam, o, lse, o2,
                    {1, H, Hkv, max_seqlen, d, cu_seqlens, num_seqs, total_tokens, scale, causal, window}, stream,
                    kWaitTimeoutNs, 0);
}

extern "C" size_t attn_diff_bwd_workspace_bytes(int B, int H, int N)
{
    if (B < 1 || H < 1 || N < 1) return 0;
    return kDiffBwdHead + (size_t)B * H * N * 2 * sizeof(float);
}

extern "C" attn_status_t attn_diff_bwd_bf16(const void* q, const void* k, const void* v, const float* lam,
                                            const void* o, const void* o2, const void* dout, const float* lse, void* dq,
                                            void* dk, void* dv, float* dlam, void* workspace, size_t workspace_bytes,
                                            int B, int H, int Hkv, int N, int d, float scale, int causal, int window,
                                            void* stream)
{
    if (B < 1 || N < 1) return ATTN_ERR_INVALID_ARG;
    const attn_status_t st = diff_sizes(H, Hkv, d, scale);
    if (st != ATTN_OK) return st;
    if (!q || !k || !v || !lam || !o || !o2 || !dout || !lse || !dq || !dk || !dv || !dlam || !workspace)
        return ATTN_ERR_INVALID_ARG;
    if (workspace_bytes < attn_diff_bwd_workspace_bytes(B, H, N)) return ATTN_ERR_INVALID_ARG;
    return diff_bwd(q, k, v, lam, o, o2, dout, lse, dq, dk, dv, dlam, workspace,
                    {B, H, Hkv, N, d, nullptr, 0, -1, scale, causal, window}, stream, kWaitTimeoutNs, 0);
}

extern "C" attn_status_t attn_diff_bwd_bf16_varlen(const void* q, const void* k, const void* v, const float* lam,
                                                   const void* o, const void* o2, const void* dout, const float* lse,
                                                   void* dq, void* dk, void* dv, float* dlam, void* workspace,
                                                   size_t workspace_bytes, const int* cu_seqlens, int num_seqs,
                                                   int max_seqlen, int total_tokens, int H, int Hkv, int d, float scale,
                                                   int causal, int window, void* stream)
{
    if (num_seqs < 1 || total_tokens < 0 || max_seqlen < 0 || max_seqlen > total_tokens) return ATTN_ERR_INVALID_ARG;
    const attn_status_t st = diff_sizes(H, Hkv, d, scale);
    if (st != ATTN_OK) return st;
    if (!dlam) return ATTN_ERR_INVALID_ARG;
    if (total_tokens == 0 || max_seqlen == 0) {          // no rows: the sum over them is 0
        if (!aligned(dlam, 4)) return ATTN_ERR_MISALIGNED;
        return cudaMemsetAsync(dlam, 0, (size_t)H * sizeof(float), static_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? ATTN_OK : ATTN_ERR_CUDA;
    }
    if (!q || !k || !v || !lam || !o || !o2 || !dout || !lse || !dq || !dk || !dv || !workspace || !cu_seqlens)
        return ATTN_ERR_INVALID_ARG;
    if (workspace_bytes < attn_diff_bwd_workspace_bytes(1, H, total_tokens)) return ATTN_ERR_INVALID_ARG;
    return diff_bwd(q, k, v, lam, o, o2, dout, lse, dq, dk, dv, dlam, workspace,
                    {1, H, Hkv, max_seqlen, d, cu_seqlens, num_seqs, total_tokens, scale, causal, window}, stream,
                    kWaitTimeoutNs, 0);
}

// ------------------------------------------------------------------ decoding over a paged cache
namespace {

// Tables of at most this many keys: a pair's tiles stay with one CTA and nothing is joined.
constexpr int kDiffDecodeWholeKeys = 384;
constexpr int kDiffDecodeMaxBatch = (1 << 19) - 1;   // decode_fp8.cuh packs a count of sequences into 19 bits

struct DiffDecodePlan {
    int cta_rows, ranges, row_groups;
};

DiffDecodePlan diff_decode_plan(int rows, int d, int sm_count)
{
    DiffDecodePlan plan;
    plan.cta_rows = diff_decode_rows(rows, d);
    plan.row_groups = (rows + plan.cta_rows - 1) / plan.cta_rows;
    const int ctas = diff_decode_ctas(d) * sm_count;
    plan.ranges = ctas / plan.row_groups > 1 ? ctas / plan.row_groups : 1;
    return plan;
}

size_t diff_decode_ws_bytes(const DiffDecodePlan& plan, int d)
{
    // per CTA: what the joining kernel has to do (16 bytes), and two parts of both maps
    return (size_t)plan.ranges * plan.row_groups * (4 + 2 * (2 * plan.cta_rows) * (2 * d + 2)) * sizeof(float);
}

attn_status_t diff_decode(const void* q, const void* k_cache, const void* v_cache, const float* lam,
                          const int* page_table, const int* seq_lens, void* o, float* lse, int B, int H, int Hkv, int nq,
                          int d, int page_size, int num_pages, int max_pages, float scale, int window, void* workspace,
                          size_t workspace_bytes, void* stream, unsigned long long timeout_ns, int withhold)
{
    if (!q || !k_cache || !v_cache || !lam || !page_table || !seq_lens || !o || !lse) return ATTN_ERR_INVALID_ARG;
    if (B < 1 || nq < 1 || num_pages < 1 || max_pages < 1) return ATTN_ERR_INVALID_ARG;
    attn_status_t st = diff_sizes(H, Hkv, d, scale);
    if (st != ATTN_OK) return st;
    if (nq > 8 || page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
        return ATTN_ERR_UNSUPPORTED;
    if ((long long)max_pages * page_size > 0x7fffffffLL || (long long)num_pages * Hkv > 0x7fffffffLL / 2 || H > 65535 ||
        (long long)B * H > 0x7fffffffLL / 2 / nq || B > kDiffDecodeMaxBatch)
        return ATTN_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lam, 4) ||
        !aligned(lse, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 16))
        return ATTN_ERR_MISALIGNED;
    DeviceInfo* dev = nullptr;
    st = device_info(&dev);
    if (st != ATTN_OK) return st;
    const int rows = H / Hkv * nq;
    const DiffDecodePlan plan = diff_decode_plan(rows, d, dev->sm_count);
    if (diff_decode_ws_bytes(plan, d) > (workspace ? workspace_bytes : 0)) return ATTN_ERR_INVALID_ARG;
    // the caches as (d, page_size, pages * 2 Hkv), boxes of one page or 64 rows of a larger one
    alignas(64) CUtensorMap mk, mv;
    const int box = page_size < 64 ? page_size : 64;
    const long long heads = 2LL * num_pages * Hkv;
    if (!encode_rows(&mk, k_cache, d, page_size, d, heads, (long long)page_size * d, box) ||
        !encode_rows(&mv, v_cache, d, page_size, d, heads, (long long)page_size * d, box))
        return ATTN_ERR_CUDA;
    DiffDecodeParams p;
    std::memset(&p, 0, sizeof(p));
    p.w.q = q;
    p.w.page_table = page_table;
    p.w.seq_lens = seq_lens;
    p.w.o = o;
    p.w.lse = lse;
    p.w.B = B;
    p.w.Hkv = Hkv;
    p.w.nq = nq;
    p.w.rows = rows;
    while ((1 << p.w.log2_ps) < page_size) ++p.w.log2_ps;
    p.w.num_pages = num_pages;
    p.w.max_pages = max_pages;
    p.w.window = window > 0 && window < max_pages * page_size ? window : 0;   // a wider one hides nothing
    p.w.c_log2 = (float)((double)scale * 1.4426950408889634);
    p.w.ws = static_cast<float*>(workspace);
    p.w.whole = max_pages * page_size <= kDiffDecodeWholeKeys ? 1 : 0;
    p.w.ranges = plan.ranges;
    p.w.row_groups = plan.row_groups;
    p.w.status = dev->status;
    p.w.timeout_ns = timeout_ns;
    p.w.withhold = (unsigned)withhold;
    p.lam = lam;
    p.H = H;
    return launch_diff_decode(mk, mv, p, d, plan.cta_rows, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" size_t attn_diff_decode_workspace_bytes(int H, int Hkv, int nq, int d)
{
    if (H < 1 || Hkv < 1 || nq < 1 || nq > 8 || H % Hkv != 0 || H > 65535 || (d != 64 && d != 128)) return 0;
    DeviceInfo* dev = nullptr;
    if (device_info(&dev) != ATTN_OK) return 0;
    return diff_decode_ws_bytes(diff_decode_plan(H / Hkv * nq, d, dev->sm_count), d);
}

extern "C" attn_status_t attn_diff_decode_bf16_paged(const void* q, const void* k_cache, const void* v_cache,
                                                     const float* lam, const int* page_table, const int* seq_lens,
                                                     void* o, float* lse, int B, int H, int Hkv, int nq, int d,
                                                     int page_size, int num_pages, int max_pages, float scale,
                                                     int window, void* workspace, size_t workspace_bytes, void* stream)
{
    return diff_decode(q, k_cache, v_cache, lam, page_table, seq_lens, o, lse, B, H, Hkv, nq, d, page_size, num_pages,
                       max_pages, scale, window, workspace, workspace_bytes, stream, kWaitTimeoutNs, 0);
}

// ------------------------------------------------------------------ abort paths
// The production kernels with one load withheld and a short limit on every wait.
static bool selftest_ok(int withheld, unsigned long long timeout_ns)
{
    return withheld >= 0 && withheld < 0x7ffffffe && timeout_ns > 0 && timeout_ns <= 2000000000ull;
}

extern "C" attn_status_t attn_selftest_diff_fwd_withheld_load(const void* q, const void* k, const void* v,
                                                             const float* lam, void* o, float* lse, int B, int H,
                                                             int Hkv, int N, int d, int causal, int withheld,
                                                             unsigned long long timeout_ns, void* stream)
{
    if (!selftest_ok(withheld, timeout_ns) || B < 1 || N < 1) return ATTN_ERR_INVALID_ARG;
    const attn_status_t st = diff_sizes(H, Hkv, d, 1.0f);
    if (st != ATTN_OK) return st;
    if (!q || !k || !v || !lam || !o || !lse) return ATTN_ERR_INVALID_ARG;
    return diff_fwd(q, k, v, lam, o, lse, nullptr,
                    {B, H, Hkv, N, d, nullptr, 0, -1, 1.0f / std::sqrt((float)d), causal, 0}, stream, timeout_ns,
                    withheld + 1);
}

extern "C" attn_status_t attn_selftest_diff_bwd_withheld_load(
    const void* q, const void* k, const void* v, const float* lam, const void* o, const void* o2, const void* dout,
    const float* lse, void* dq, void* dk, void* dv, float* dlam, void* workspace, size_t workspace_bytes, int B, int H,
    int Hkv, int N, int d, int causal, int withheld, unsigned long long timeout_ns, void* stream)
{
    if (!selftest_ok(withheld, timeout_ns) || B < 1 || N < 1) return ATTN_ERR_INVALID_ARG;
    const attn_status_t st = diff_sizes(H, Hkv, d, 1.0f);
    if (st != ATTN_OK) return st;
    if (!q || !k || !v || !lam || !o || !o2 || !dout || !lse || !dq || !dk || !dv || !dlam || !workspace ||
        workspace_bytes < attn_diff_bwd_workspace_bytes(B, H, N))
        return ATTN_ERR_INVALID_ARG;
    return diff_bwd(q, k, v, lam, o, o2, dout, lse, dq, dk, dv, dlam, workspace,
                    {B, H, Hkv, N, d, nullptr, 0, -1, 1.0f / std::sqrt((float)d), causal, 0}, stream, timeout_ns,
                    withheld + 1);
}

extern "C" attn_status_t attn_selftest_diff_decode_withheld_load(
    const void* q, const void* k_cache, const void* v_cache, const float* lam, const int* page_table,
    const int* seq_lens, void* o, float* lse, int B, int H, int Hkv, int nq, int d, int page_size, int num_pages,
    int max_pages, void* workspace, size_t workspace_bytes, int withheld, unsigned long long timeout_ns, void* stream)
{
    if (!selftest_ok(withheld, timeout_ns) || d < 1) return ATTN_ERR_INVALID_ARG;
    return diff_decode(q, k_cache, v_cache, lam, page_table, seq_lens, o, lse, B, H, Hkv, nq, d, page_size, num_pages,
                       max_pages, 1.0f / std::sqrt((float)d), 0, workspace, workspace_bytes, stream, timeout_ns,
                       withheld + 1);
}
