// C ABI entry points that train the tile predictor: the pooled teacher, the scores with a relative position
// bias, the distillation loss and the gradients. Argument checks and launches; the kernels live in
// teacher.cuh, train_gemm.cuh, bias.cuh and distill.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <string>

#include "veda_internal.h"
#include "bias.cuh"
#include "distill.cuh"
#include "teacher.cuh"
#include "train_gemm.cuh"

using namespace veda;

namespace {

constexpr int kMaxTrainTiles = 16384;  // the widest row veda_select takes

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
size_t round256(size_t b) { return (b + 255) & ~size_t(255); }

// A buffer of a call; `base` may be null (no buffer, no overlap)
struct Span {
    const char* name;
    const void* base;
    int64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.base), y = reinterpret_cast<uintptr_t>(b.base);
    return x && y && x < y + uint64_t(b.bytes) && y < x + uint64_t(a.bytes);
}

template <class F>
int guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        return VEDA_ERR_CUDA;  // out of host memory while a message was made
    }
}

int check_heads(const char* who, int32_t n_heads, int32_t dim) {
    if (dim != 64 && dim != 128) return fail(VEDA_ERR_INVALID, std::string(who) + ": head_dim must be 64 or 128");
    if (n_heads <= 0) return fail(VEDA_ERR_INVALID, std::string(who) + ": n_heads must be positive");
    return VEDA_OK;
}

int check_size(const char* who, const veda_layout* layout, int32_t n_heads) {
    if (layout->desc.n_video > kMaxTrainTiles || n_heads > 65535)
        return fail(VEDA_ERR_UNSUPPORTED, std::string(who) + ": at most 16384 video tiles and 65535 heads");
    return VEDA_OK;
}

int classes_of(const char* who, const veda_bias_spec* spec, BiasClasses* out) {
    if (!spec) return fail(VEDA_ERR_INVALID, std::string(who) + ": the bias specification is NULL");
    int64_t buckets = 1;
    for (int a = 0; a < 3; ++a) {
        const int reach = spec->reach[a], far = spec->far_tiles[a], exact = (reach + 1) / 2, wide = reach - exact;
        if (reach < 1 || reach > kBiasMaxReach)
            return fail(VEDA_ERR_INVALID, std::string(who) + ": reach must lie in [1, 16] on every axis");
        if (far <= exact || far > 32767)
            return fail(VEDA_ERR_INVALID, std::string(who) + ": far must lie in ((reach + 1) / 2, 32767] on every axis");
        out->reach[a] = reach;
        for (int c = 0; c < kBiasMaxReach; ++c) out->starts[a][c] = c;
        for (int m = 1; exact + m < reach; ++m) {
            unsigned __int128 bound = 1;  // exact^(wide - m) far^m < 2^120
            for (int k = 0; k < wide; ++k) bound *= unsigned(k < m ? far : exact);
            int lo = exact, hi = far;     // the smallest distance whose wide-th power reaches the bound
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                unsigned __int128 p = 1;
                for (int k = 0; k < wide; ++k) p *= unsigned(mid);
                if (p >= bound) hi = mid; else lo = mid + 1;
            }
            out->starts[a][exact + m] = lo;
        }
        buckets *= 2 * reach - 1;
    }
    buckets += 2;
    if (buckets > kBiasMaxBuckets)
        return fail(VEDA_ERR_UNSUPPORTED, std::string(who) + ": at most 4096 buckets");
    out->buckets = int(buckets);
    return VEDA_OK;
}

// Key runs per group of query tiles. A unit costs its key pairs plus about one and a half pairs' time to load Q and
// to fill and drain the pipeline; the runs are the number that makes the busiest CTA's sum least.
int teacher_runs(int64_t groups, int pairs, int sms) {
    int best = 1;
    double least = 1e300;
    for (int c = 1; c <= std::min(pairs, 64); ++c) {
        const double cost = double((groups * c + sms - 1) / sms) * ((pairs + c - 1) / c + 1.5);
        if (cost < least * 0.995) {
            least = cost;
            best = c;
        }
    }
    return best;
}

template <int D>
int launch_teacher(const teacher::Maps& m, const teacher::Args& a, const DeviceInfo& di, cudaStream_t s) {
    static std::atomic<bool> set[kMaxDevices];
    if (!set[di.ordinal].load()) {
        cudaError_t e = cudaFuncSetAttribute(teacher::teacher_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(teacher::Cfg<D>::kSmem));
        if (e != cudaSuccess)
            return fail(VEDA_ERR_CUDA, std::string("cudaFuncSetAttribute(teacher_kernel): ") + cudaGetErrorString(e));
        set[di.ordinal].store(true);
    }
    teacher::teacher_kernel<D><<<unsigned(std::min(a.units, di.sms)), teacher::kThreads, teacher::Cfg<D>::kSmem, s>>>(m, a);
    return launch_status("teacher_kernel");
}

// [batch][rows][K] with rows of K innermost (cols: [batch][K][rows]), densely packed
train::Operand operand(const float* base, int rows, int K, bool cols) {
    const int64_t stride = cols ? rows : K;
    return {base, int64_t(rows) * K, stride, rows, cols ? train::kCols : train::kRows, stride % 4 == 0};
}

// the operand's map, or its four
int operand_maps(CUtensorMap* m, const train::Operand& o, int K, int batches) {
    if (o.dense)
        return o.layout == train::kCols ? make_f32_cols_map(m, o.base, o.rows, K, batches) : make_f32_map(m, o.base, K, o.rows, batches);
    const int64_t rows = int64_t(batches) * (o.layout == train::kCols ? K : o.rows);
    for (int b = 0; b < 4; ++b)
        if (int rc = o.layout == train::kCols
                         ? make_f32_fourth_rows_map(m + b, o.base, o.stride, rows, b, train::kQuadCols, train::kQuadK)
                         : make_f32_fourth_rows_map(m + b, o.base, o.stride, rows, b, train::kQuadWidth, train::kQuadRows))
            return rc;
    return VEDA_OK;
}

constexpr int kSplitUnits = 148, kSplitSlices = 4, kJoinSlices = 6;
constexpr size_t kSplitBytes = size_t(kSplitUnits) * train::kBM * train::kBN * sizeof(float);  // parts of split tiles

// Tiles past whole rounds of CTAs are cut along K into as many parts as CTAs are left, of at least kSplitSlices slices,
// when that shortens the last round by more than joining the parts takes (about kJoinSlices slices' time). 819 tiles,
// D 128, both gradients in runs of a few milliseconds: 24 heads 96 -> 93 us, 8 heads 50 -> 46, 1 head 46 -> 24 (now 97 with
// 24 heads: hi_part's bound). More than one part takes a launch more.
int parts_along_k(int64_t tiles, int K, int sms) {
    const int nk = (K + train::kBK - 1) / train::kBK, rest = int(tiles % sms);
    const int parts = rest ? std::min(std::min(sms, kSplitUnits) / rest, nk / kSplitSlices) : 1;
    return parts < 2 || nk - (nk + parts - 1) / parts < kJoinSlices ? 1 : parts;
}
int64_t tiles_of(int sets, int batches, int M, int N) {
    return int64_t(sets) * batches * ((M + train::kBM - 1) / train::kBM) * ((N + train::kBN - 1) / train::kBN);
}

// `after`: the launch before it on the stream is one of this call's, and its start may overlap that one's end
template <int kParts>
int launch_gemm(const char* what, train::Args a, const BiasExpand& expand, bool after, const DeviceInfo& di, cudaStream_t s) {
    static std::atomic<bool> set[kMaxDevices];
    if (!set[di.ordinal].load()) {
        cudaError_t e = cudaFuncSetAttribute(train::gemm_kernel<kParts>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(train::kSmem));
        if (e != cudaSuccess)
            return fail(VEDA_ERR_CUDA, std::string("cudaFuncSetAttribute(train gemm_kernel): ") + cudaGetErrorString(e));
        set[di.ordinal].store(true);
    }
    a.tiles_m = (a.M + train::kBM - 1) / train::kBM;
    a.tiles_n = (a.N + train::kBN - 1) / train::kBN;
    const int64_t tiles = tiles_of(a.n_sets, a.nb, a.M, a.N);
    if (tiles > INT32_MAX - kSplitUnits) return fail(VEDA_ERR_UNSUPPORTED, std::string(what) + ": too many tiles for one launch");
    const int rest = int(tiles % di.sms);
    a.parts = a.partial ? parts_along_k(tiles, a.K, di.sms) : 1;
    a.full = int(tiles) - (a.parts > 1 ? rest : 0);
    a.n_units = a.full + (a.parts > 1 ? rest * a.parts : 0);
    a.timeout_ns = wait_timeout_ns();
    a.err = di.err;
    train::Maps m{};
    for (int i = 0; i < a.n_sets; ++i) {
        if (int rc = operand_maps(&m.a[i], a.set[i].a, a.K, a.nb)) return rc;
        if (int rc = operand_maps(m.b[i], a.set[i].b, a.K, a.nb)) return rc;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(std::min(a.n_units, di.sms)));
    cfg.blockDim = dim3(train::threads_of(kParts));
    cfg.dynamicSmemBytes = train::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute overlap{};
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &overlap;
    cfg.numAttrs = after ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, train::gemm_kernel<kParts>, m, a, expand);
    if (e != cudaSuccess) return fail(VEDA_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
    if (int rc = launch_status(what)) return rc;
    if (a.parts == 1) return VEDA_OK;
    cfg.gridDim = dim3(train::kBM * train::kBN / 1024, unsigned(rest));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, train::join_kernel, a);
    if (e != cudaSuccess) return fail(VEDA_ERR_CUDA, std::string(what) + " (join): " + cudaGetErrorString(e));
    return launch_status(what);
}

template <int kPer, int kWarps>
int launch_distill(const DistillArgs& a, cudaStream_t s) {
    const int64_t ctas = kWarps == 1 ? (a.rows + 3) / 4 : a.rows;  // at most 65535 * 16384, under 2^31
    distill_kernel<kPer, kWarps><<<unsigned(ctas), kWarps == 1 ? 128 : 32 * kWarps, 0, s>>>(a);
    return launch_status("distill_kernel");
}

// Query rows of one chunk of the bias gradient's sums: with all heads one to three CTAs (six of the kernel without offset
// sums) for each of 148 SMs, but not fewer than eight rows, which a chunk's own start and end cost. How many is a table by
// the row length, from what was measured with these kernels' registers, not what could be resident: at 128 tiles ten CTAs
// would fit, at 1,100 four; and shared memory is not looked at, which lets in one CTA of 16 x 16 x 16 tiles (116 KB of
// offset sums) where the table says two. Three against two: 819 tiles, 24 heads 28 and 32 us, 480 tiles (a CTA too many) 24
// and 16, 1860 tiles 110 and 82; two against one: 3720 tiles, 8 heads 103 and 130, 7320 tiles, 4 heads 231 and 205. The
// kernel without offset sums is bound by latency: 14,880 tiles, 2 heads 8.6, 3.2, 2.8 ms with one, three, six.
int bias_chunk_rows(int n, int n_heads) {
    const int resident = n <= 1024 ? (n <= 416 || n > 512 ? 3 : 2) : n <= 4096 ? 2 : n <= 8192 ? 1 : 6;
    const int chunks = std::max(1, std::min(148 * resident / std::max(n_heads, 1), (n + 7) / 8));
    return std::max(1, (n + chunks - 1) / chunks);
}
int bias_chunks(int n, int n_heads) {
    const int rows = bias_chunk_rows(n, n_heads);
    return (n + rows - 1) / rows;
}

constexpr int kBiasMaxSmem = 227 * 1024;
// the sums, the warps' cross-span sums, and a query of 8 bytes per row
size_t bias_smem(const BiasBackwardArgs& a) {
    return (size_t(a.offsets) + 32 + 1) / 2 * 8 + size_t(a.rows_per_chunk) * 8;
}

template <int kPer, bool kOneSpan>
int launch_bias_backward(const BiasBackwardArgs& a, int chunks, int n_heads, const DeviceInfo& di, cudaStream_t s) {
    static std::atomic<bool> set[kMaxDevices];
    if (!set[di.ordinal].load()) {
        cudaError_t e = cudaFuncSetAttribute(bias_backward_kernel<kPer, kOneSpan>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBiasMaxSmem);
        if (e != cudaSuccess)
            return fail(VEDA_ERR_CUDA, std::string("cudaFuncSetAttribute(bias_backward_kernel): ") + cudaGetErrorString(e));
        set[di.ordinal].store(true);
    }
    const int threads = std::max(128, ((a.n + kPer - 1) / kPer + 31) / 32 * 32);
    bias_backward_kernel<kPer, kOneSpan><<<dim3(chunks, n_heads), threads, bias_smem(a), s>>>(a);
    return launch_status("bias_backward_kernel");
}

// (the limit is the function's, shared by all host threads: it is set once, for the widest row)
int launch_bias_wide(const BiasBackwardArgs& a, int chunks, int n_heads, const DeviceInfo& di, cudaStream_t s) {
    static std::atomic<bool> set[kMaxDevices];
    if (!set[di.ordinal].load()) {
        cudaError_t e = cudaFuncSetAttribute(bias_backward_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kMaxTrainTiles * int(sizeof(float)));
        if (e != cudaSuccess)
            return fail(VEDA_ERR_CUDA, std::string("cudaFuncSetAttribute(bias_backward_wide_kernel): ") + cudaGetErrorString(e));
        set[di.ordinal].store(true);
    }
    bias_backward_wide_kernel<<<dim3(chunks, n_heads), 256, a.n * sizeof(float), s>>>(a);
    return launch_status("bias_backward_wide_kernel");
}

template <int kPer>
int launch_bias(bool one_span, const BiasBackwardArgs& a, int chunks, int n_heads, const DeviceInfo& di, cudaStream_t s) {
    return one_span ? launch_bias_backward<kPer, true>(a, chunks, n_heads, di, s)
                    : launch_bias_backward<kPer, false>(a, chunks, n_heads, di, s);
}

}  // namespace

extern "C" int veda_bias_buckets(const veda_bias_spec* spec, int32_t* n_buckets) {
    return guarded([&] {
        clear_error();
        if (!n_buckets) return fail(VEDA_ERR_INVALID, "veda_bias_buckets: NULL argument");
        BiasClasses b;
        if (int rc = classes_of("veda_bias_buckets", spec, &b)) return rc;
        *n_buckets = b.buckets;
        return VEDA_OK;
    });
}

extern "C" int veda_bias_index(const veda_layout* layout, const veda_bias_spec* spec, int32_t* index) {
    return guarded([&] {
        clear_error();
        if (!layout || !index) return fail(VEDA_ERR_INVALID, "veda_bias_index: NULL argument");
        BiasClasses b;
        if (int rc = classes_of("veda_bias_index", spec, &b)) return rc;
        const int64_t n = layout->desc.n_video;
        const int32_t* pos = layout->tile_pos.data();
        for (int64_t i = 0; i < n; ++i)
            for (int64_t j = 0; j < n; ++j) {
                const int32_t *q = pos + 4 * i, *k = pos + 4 * j;
                index[i * n + j] = k[0] < q[0]   ? b.buckets - 2
                                   : k[0] > q[0] ? b.buckets - 1
                                                 : bias_bucket(b, k[1] - q[1], k[2] - q[2], k[3] - q[3]);
            }
        return VEDA_OK;
    });
}

extern "C" int veda_teacher(const veda_layout* layout, const void* q_t, const void* k_t, int32_t n_heads, int32_t dim,
                            const float* row_lse, float* teacher, void* stream) {
    return guarded([&] {
        clear_error();
        if (!layout || !q_t || !k_t || !teacher) return fail(VEDA_ERR_INVALID, "veda_teacher: NULL argument");
        if (int rc = check_heads("veda_teacher", n_heads, dim)) return rc;
        if (!aligned16(q_t) || !aligned16(k_t) || !aligned16(row_lse) || !aligned16(teacher))
            return fail(VEDA_ERR_INVALID, "veda_teacher: buffers need 16-byte alignment");
        if (int rc = check_size("veda_teacher", layout, n_heads)) return rc;
        DeviceInfo di;
        if (int rc = current_device(&di)) return rc;
        const DeviceCopy* dc;
        if (int rc = layout_on_device(layout, &dc)) return rc;
        const veda_layout_desc& d = layout->desc;
        if (int64_t(n_heads) * d.n_slots > INT32_MAX)
            return fail(VEDA_ERR_UNSUPPORTED, "veda_teacher: more than 2^31 tile-ordered rows");
        teacher::Maps m;
        if (int rc = make_bf16_rows_map(&m.q, q_t, n_heads * d.n_slots, dim)) return rc;
        if (int rc = make_bf16_rows_map(&m.k, k_t, n_heads * d.n_slots, dim)) return rc;
        teacher::Args a{};
        a.valid_count = dc->valid_count;
        a.perm = dc->perm;
        a.lse = row_lse;
        a.out = teacher;
        a.seq_len = d.seq_len;
        a.n = d.n_video;
        a.n_tiles = d.n_tiles;
        a.groups = (a.n + 1) / 2;
        a.pairs = (a.n + 1) / 2;
        a.runs = teacher_runs(int64_t(n_heads) * a.groups, a.pairs, di.sms);
        if (int64_t(n_heads) * a.groups * a.runs > INT32_MAX)
            return fail(VEDA_ERR_UNSUPPORTED, "veda_teacher: too many work units for one launch");
        a.units = n_heads * a.groups * a.runs;
        a.scale = float(1.0 / std::sqrt(double(dim)));
        a.timeout_ns = wait_timeout_ns();
        a.err = di.err;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        return dim == 128 ? launch_teacher<128>(m, a, di, s) : launch_teacher<64>(m, a, di, s);
    });
}

extern "C" size_t veda_score_bias_workspace_bytes(const veda_layout* layout, int32_t n_heads, int32_t dim) {
    if (!layout || n_heads <= 0 || dim <= 0) return 0;
    return kSplitBytes + round256(size_t(n_heads) * size_t(layout->bias_offsets + 2) * sizeof(float));
}

extern "C" int veda_score_bias_launches(const veda_layout* layout, int32_t n_heads, int32_t dim, int32_t* launches) {
    return guarded([&] {
        clear_error();
        if (!layout || !launches) return fail(VEDA_ERR_INVALID, "veda_score_bias_launches: NULL argument");
        if (int rc = check_heads("veda_score_bias_launches", n_heads, dim)) return rc;
        if (int rc = check_size("veda_score_bias_launches", layout, n_heads)) return rc;
        DeviceInfo di;
        if (int rc = current_device(&di)) return rc;
        // the projections, cut or not, and the logits
        *launches = 2 + (parts_along_k(tiles_of(2, n_heads, dim, layout->desc.n_video), 3 * dim, di.sms) > 1);
        return VEDA_OK;
    });
}

extern "C" int veda_score_bias(const veda_layout* layout, const float* feats_q, const float* feats_k, int32_t n_heads,
                               int32_t dim, const float* proj_q, const float* proj_k, const veda_bias_spec* spec,
                               const float* bias, float* hats, void* workspace, size_t workspace_bytes, float* scores,
                               void* stream) {
    return guarded([&] {
        clear_error();
        if (!layout || !feats_q || !feats_k || !proj_q || !proj_k || !hats || !workspace || !scores || !spec != !bias)
            return fail(VEDA_ERR_INVALID, "veda_score_bias: NULL argument (spec and bias go together)");
        if (int rc = check_heads("veda_score_bias", n_heads, dim)) return rc;
        if (workspace_bytes < veda_score_bias_workspace_bytes(layout, n_heads, dim))
            return fail(VEDA_ERR_INVALID, "veda_score_bias: workspace smaller than veda_score_bias_workspace_bytes()");
        for (const void* p : {(const void*)feats_q, (const void*)feats_k, (const void*)proj_q, (const void*)proj_k,
                              (const void*)bias, (const void*)hats, (const void*)workspace, (const void*)scores})
            if (!aligned16(p)) return fail(VEDA_ERR_INVALID, "veda_score_bias: buffers need 16-byte alignment");
        if (int rc = check_size("veda_score_bias", layout, n_heads)) return rc;
        BiasClasses b;
        if (spec)
            if (int rc = classes_of("veda_score_bias", spec, &b)) return rc;
        DeviceInfo di;
        if (int rc = current_device(&di)) return rc;
        const DeviceCopy* dc;
        if (int rc = layout_on_device(layout, &dc)) return rc;
        const int n = layout->desc.n_video;
        const int offsets = layout->bias_offsets;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        float* table = static_cast<float*>(workspace) + kSplitBytes / sizeof(float);  // behind the parts of split tiles
        BiasExpand expand{};
        if (bias)
            expand = {bias, table, float(std::sqrt(double(dim))), reinterpret_cast<const int4*>(dc->span_grid),
                      int(layout->span_grid.size() / 4), offsets, n_heads, b};
        const int64_t nd = int64_t(n) * dim;
        // hats[tile][d], both sides in one launch, then scores[query][key]
        train::Args p{};
        p.n_sets = 2;
        p.nb = n_heads;
        p.M = dim;
        p.N = n;
        p.K = 3 * dim;
        p.scale = 1.f;
        p.identity = 1;
        p.partial = static_cast<float*>(workspace);
        for (int side = 0; side < 2; ++side) {
            const float* f = side ? feats_k : feats_q;
            p.set[side] = {operand(side ? proj_k : proj_q, dim, 3 * dim, true), operand(f, n, 3 * dim, false),
                           hats + side * n_heads * nd};
        }
        if (int rc = launch_gemm<4>("veda_score_bias (projections)", p, expand, false, di, s)) return rc;
        train::Args l{};
        l.n_sets = 1;
        l.nb = n_heads;
        l.M = l.N = n;
        l.K = dim;
        l.scale = float(1.0 / std::sqrt(double(dim)));
        l.set[0] = {operand(hats + n_heads * nd, n, dim, false), operand(hats, n, dim, false), scores};
        l.one_span = layout->span_grid.size() == 4;
        if (bias) l.table = table;
        l.tile_num = reinterpret_cast<const int4*>(dc->tile_num);
        l.table_stride = offsets + 2;
        l.offsets = offsets;
        return launch_gemm<4>("veda_score_bias (logits)", l, BiasExpand{}, true, di, s);
    });
}

extern "C" size_t veda_bias_backward_workspace_bytes(const veda_layout* layout, int32_t n_heads, const veda_bias_spec* spec) {
    BiasClasses b;
    if (!layout || n_heads <= 0 || guarded([&] { return classes_of("veda_bias_backward_workspace_bytes", spec, &b); })) return 0;
    return round256(size_t(n_heads) * bias_chunks(layout->desc.n_video, n_heads) * size_t(b.buckets) * sizeof(float));
}

extern "C" int veda_bias_backward(const veda_layout* layout, const float* d_scores, int32_t n_heads,
                                  const veda_bias_spec* spec, void* workspace, size_t workspace_bytes, float* d_bias,
                                  void* stream) {
    return guarded([&] {
        clear_error();
        if (!layout || !d_scores || !workspace || !d_bias) return fail(VEDA_ERR_INVALID, "veda_bias_backward: NULL argument");
        if (n_heads <= 0) return fail(VEDA_ERR_INVALID, "veda_bias_backward: n_heads must be positive");
        BiasBackwardArgs a{};
        if (int rc = classes_of("veda_bias_backward", spec, &a.b)) return rc;
        if (workspace_bytes < veda_bias_backward_workspace_bytes(layout, n_heads, spec))
            return fail(VEDA_ERR_INVALID, "veda_bias_backward: workspace smaller than veda_bias_backward_workspace_bytes()");
        if (!aligned16(d_scores) || !aligned16(workspace) || !aligned16(d_bias))
            return fail(VEDA_ERR_INVALID, "veda_bias_backward: buffers need 16-byte alignment");
        if (int rc = check_size("veda_bias_backward", layout, n_heads)) return rc;
        DeviceInfo di;
        if (int rc = current_device(&di)) return rc;
        const DeviceCopy* dc;
        if (int rc = layout_on_device(layout, &dc)) return rc;
        a.d_scores = d_scores;
        a.tile_pos = reinterpret_cast<const int4*>(dc->tile_pos);
        a.span_grid = reinterpret_cast<const int4*>(dc->span_grid);
        a.partial = static_cast<float*>(workspace);
        a.n = layout->desc.n_video;
        a.tile_num = reinterpret_cast<const int4*>(dc->tile_num);
        a.n_spans = int(layout->span_grid.size() / 4);
        a.offsets = layout->bias_offsets;
        a.rows_per_chunk = bias_chunk_rows(a.n, n_heads);
        const int chunks = bias_chunks(a.n, n_heads);
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        int rc;
        if (bias_smem(a) > size_t(kBiasMaxSmem) || a.n > 8192) {
            rc = launch_bias_wide(a, chunks, n_heads, di, s);
        } else {
            const bool one = a.n_spans == 1;
            rc = a.n <= 512    ? launch_bias<1>(one, a, chunks, n_heads, di, s)
                 : a.n <= 1024 ? launch_bias<2>(one, a, chunks, n_heads, di, s)
                 : a.n <= 2048 ? launch_bias<4>(one, a, chunks, n_heads, di, s)
                 : a.n <= 4096 ? launch_bias<8>(one, a, chunks, n_heads, di, s)
                               : launch_bias<16>(one, a, chunks, n_heads, di, s);
        }
        if (rc) return rc;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(unsigned(a.b.buckets + 127) / 128, unsigned(n_heads));
        cfg.blockDim = dim3(128);
        cfg.stream = s;
        cudaLaunchAttribute overlap{};
        overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        overlap.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &overlap;
        cfg.numAttrs = 1;
        cudaError_t e = cudaLaunchKernelEx(&cfg, bias_reduce_kernel, static_cast<const float*>(a.partial), d_bias, chunks, int(a.b.buckets));
        if (e != cudaSuccess) return fail(VEDA_ERR_CUDA, std::string("bias_reduce_kernel: ") + cudaGetErrorString(e));
        return launch_status("bias_reduce_kernel");
    });
}

extern "C" int veda_distill(const veda_layout* layout, const float* scores, int32_t n_heads, const int32_t* t_idx,
                            const float* t_val, const int32_t* t_cnt, int32_t width, int32_t by_column, float tau,
                            const float* row_weight, float* loss, float* d_scores, void* stream) {
    return guarded([&] {
        clear_error();
        if (!layout || !scores || !t_idx || !t_val || !t_cnt || !loss) return fail(VEDA_ERR_INVALID, "veda_distill: NULL argument");
        if (n_heads <= 0 || width <= 0) return fail(VEDA_ERR_INVALID, "veda_distill: n_heads and width must be positive");
        if (!(tau >= 1e-30f && tau <= 1e30f)) return fail(VEDA_ERR_INVALID, "veda_distill: tau must lie in [1e-30, 1e30]");
        for (const void* p : {(const void*)scores, (const void*)t_idx, (const void*)t_val, (const void*)t_cnt,
                              (const void*)row_weight, (const void*)loss, (const void*)d_scores})
            if (!aligned16(p)) return fail(VEDA_ERR_INVALID, "veda_distill: buffers need 16-byte alignment");
        if (int rc = check_size("veda_distill", layout, n_heads)) return rc;
        DistillArgs a{};
        a.n = layout->desc.n_video;
        a.rows = int64_t(n_heads) * a.n;
        const int64_t row = 4 * a.rows, square = row * a.n, list = row * width;
        const Span l{"loss", loss, row}, d{"d_scores", d_scores, square};
        for (const Span& in : {Span{"scores", scores, square}, Span{"t_idx", t_idx, list}, Span{"t_val", t_val, by_column ? square : list},
                               Span{"t_cnt", t_cnt, row}, Span{"row_weight", row_weight, row}})
            for (const Span& out : {l, d})
                if (overlap(out, in))
                    return fail(VEDA_ERR_INVALID, std::string("veda_distill: ") + out.name + " must not overlap " + in.name);
        if (overlap(d, l)) return fail(VEDA_ERR_INVALID, "veda_distill: d_scores must not overlap loss");
        DeviceInfo di;
        if (int rc = current_device(&di)) return rc;
        a.scores = scores;
        a.t_idx = t_idx;
        a.t_val = t_val;
        a.t_cnt = t_cnt;
        a.row_weight = row_weight;
        a.loss = loss;
        a.d_scores = d_scores;
        a.width = width;
        a.n_tiles = layout->desc.n_tiles;
        a.by_column = by_column;
        a.inv_tau = 1.f / tau;
        a.err = di.err;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        // 32 columns a thread at most; a warp's own variants in steps of four, so that few loads fall past the row
        switch (a.n <= 1024 ? (a.n + 127) / 128 : a.n <= 2048 ? 9 : a.n <= 4096 ? 10 : a.n <= 8192 ? 11 : 12) {
            case 1: return launch_distill<4, 1>(a, st);
            case 2: return launch_distill<8, 1>(a, st);
            case 3: return launch_distill<12, 1>(a, st);
            case 4: return launch_distill<16, 1>(a, st);
            case 5: return launch_distill<20, 1>(a, st);
            case 6: return launch_distill<24, 1>(a, st);
            case 7: return launch_distill<28, 1>(a, st);
            case 8: return launch_distill<32, 1>(a, st);
            case 9: return launch_distill<32, 2>(a, st);
            case 10: return launch_distill<32, 4>(a, st);
            case 11: return launch_distill<32, 8>(a, st);
            default: return launch_distill<32, 16>(a, st);
        }
    });
}

extern "C" size_t veda_score_backward_workspace_bytes(const veda_layout* layout, int32_t n_heads, int32_t dim) {
    if (!layout || n_heads <= 0 || dim <= 0) return 0;
    return kSplitBytes + round256(2 * size_t(n_heads) * size_t(layout->desc.n_video) * size_t(dim) * sizeof(float));
}

extern "C" int veda_score_backward(const veda_layout* layout, const float* feats_q, const float* feats_k, int32_t n_heads,
                                   int32_t dim, const float* hats, const float* d_scores, float* d_proj_q,
                                   float* d_proj_k, void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&] {
        clear_error();
        if (!layout || !feats_q || !feats_k || !hats || !d_scores || !d_proj_q || !d_proj_k || !workspace)
            return fail(VEDA_ERR_INVALID, "veda_score_backward: NULL argument");
        if (int rc = check_heads("veda_score_backward", n_heads, dim)) return rc;
        if (workspace_bytes < veda_score_backward_workspace_bytes(layout, n_heads, dim))
            return fail(VEDA_ERR_INVALID, "veda_score_backward: workspace smaller than veda_score_backward_workspace_bytes()");
        for (const void* p : {(const void*)feats_q, (const void*)feats_k, (const void*)hats, (const void*)d_scores,
                              (const void*)d_proj_q, (const void*)d_proj_k, (const void*)workspace})
            if (!aligned16(p)) return fail(VEDA_ERR_INVALID, "veda_score_backward: buffers need 16-byte alignment");
        if (int rc = check_size("veda_score_backward", layout, n_heads)) return rc;
        DeviceInfo di;
        if (int rc = current_device(&di)) return rc;
        const int n = layout->desc.n_video;
        const int64_t nd = int64_t(n) * dim;
        float* dx = static_cast<float*>(workspace) + kSplitBytes / sizeof(float);  // behind the parts of split tiles
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const float c = float(1.0 / std::sqrt(double(dim)));
        // dq_hat[i][d] = c sum_j dS[i][j] k_hat[j][d] and dk_hat[j][d] = c sum_i dS[i][j] q_hat[i][d], then
        // dP[f][d] = sum_i feats[i][f] dx_hat[i][d]; both sides in one launch
        train::Args x{}, p{};
        x.n_sets = p.n_sets = 2;
        x.nb = p.nb = n_heads;
        x.M = p.M = dim;
        x.N = x.K = p.K = n;
        p.N = 3 * dim;
        x.scale = c;
        p.scale = 1.f;
        x.partial = p.partial = static_cast<float*>(workspace);
        for (int side = 0; side < 2; ++side) {
            x.set[side] = {operand(hats + (side ? 0 : n_heads * nd), dim, n, true), operand(d_scores, n, n, side == 1),
                           dx + side * n_heads * nd};
            p.set[side] = {operand(dx + side * n_heads * nd, dim, n, true), operand(side ? feats_k : feats_q, 3 * dim, n, true),
                           side ? d_proj_k : d_proj_q};
        }
        if (int rc = launch_gemm<2>("veda_score_backward (projected features)", x, BiasExpand{}, false, di, s)) return rc;
        return launch_gemm<2>("veda_score_backward (projections)", p, BiasExpand{}, true, di, s);
    });
}
