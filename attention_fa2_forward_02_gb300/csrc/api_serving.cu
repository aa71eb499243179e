// api_serving.cu - the C ABI of the rotary positions, the paged key-value cache and the
// attention that reads it: argument validation, then one launch function each.
#include <math.h>

#include <utility>

#include "fa2.h"
#include "internal.h"

namespace fa2 {
namespace {

constexpr int64_t kMaxLen = (int64_t)1 << 30;
constexpr int64_t kMaxGrid = 65535;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether elements of a strided tensor (innermost: `inner` contiguous ones) never share memory:
// taken by growing stride, each dimension steps past what the smaller ones span.
bool rows_apart(const int64_t* sizes, const int64_t* strides, int dims, int64_t inner) {
    int order[3] = {0, 1, 2};  // dims <= 3
    for (int i = 1; i < dims; ++i)
        for (int j = i; j > 0 && strides[order[j]] < strides[order[j - 1]]; --j) std::swap(order[j], order[j - 1]);
    __int128 span = inner;
    for (int i = 0; i < dims; ++i) {
        const int k = order[i];
        if (sizes[k] <= 1) continue;
        if (strides[k] < span) return false;
        span += (__int128)strides[k] * (sizes[k] - 1);
    }
    return true;
}

// Strides whose products with the sizes stay far inside 63 bits.
bool strides_ok(const int64_t* strides, int n) {
    for (int i = 0; i < n; ++i)
        if (strides[i] < 0 || strides[i] > ((int64_t)1 << 40)) return false;
    return true;
}

fa2_status rope_call(const void* x, void* y, const int32_t* positions, int64_t position_stride, const double* inv_freq,
                     int64_t b, int64_t h, int64_t n, int32_t head_dim, int32_t rot_dim, const int64_t* xs,
                     const int64_t* ys, int32_t interleaved, float magnitude, fa2_dtype dtype, void* stream, bool backward) {
    if (!x || !y || !inv_freq || !xs || !ys) return FA2_ERR_INVALID_ARG;
    if (b <= 0 || h <= 0 || n <= 0 || head_dim <= 0 || rot_dim <= 0) return FA2_ERR_INVALID_ARG;
    if (dtype != FA2_DTYPE_F32 && dtype != FA2_DTYPE_F16 && dtype != FA2_DTYPE_BF16) return FA2_ERR_INVALID_ARG;
    if (rot_dim % 2 != 0 || rot_dim > head_dim || !isfinite(magnitude) || position_stride < 0 || !strides_ok(xs, 3) ||
        !strides_ok(ys, 3))
        return FA2_ERR_INVALID_ARG;
    if (head_dim > 1024 || n > kMaxLen || b > INT32_MAX || h > INT32_MAX || b * h > INT32_MAX) return FA2_ERR_UNSUPPORTED;
    const int64_t sizes[3] = {b, h, n};
    if (!rows_apart(sizes, ys, 3, head_dim)) return FA2_ERR_INVALID_ARG;
    if (x == y)
        for (int i = 0; i < 3; ++i)
            if (sizes[i] > 1 && xs[i] != ys[i]) return FA2_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(inv_freq, 8) || !aligned(positions, 4)) return FA2_ERR_MISALIGNED;
    RopeParams p{};
    p.x = x; p.y = y; p.positions = positions; p.position_stride = position_stride; p.inv_freq = inv_freq;
    p.b = b; p.h = h; p.n = n; p.d = head_dim; p.rot = rot_dim;
    for (int i = 0; i < 3; ++i) {  // a dimension of one element has no stride
        p.xs[i] = sizes[i] > 1 ? xs[i] : 0;
        p.ys[i] = sizes[i] > 1 ? ys[i] : 0;
    }
    p.interleaved = interleaved != 0; p.backward = backward; p.magnitude = magnitude; p.dtype = (int)dtype;
    return launch_rope(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA2_OK : FA2_ERR_CUDA;
}

// Checks shared by the cache's calls, and the kernels' view of the cache.
fa2_status paged(const fa2_kv_cache* c, const int32_t* table, int64_t table_stride, int64_t pages_per_seq,
                 const int32_t* lens, int64_t batch, fa2_dtype dtype, PagedParams* out) {
    if (!c || !c->k || !c->v || !table || !lens) return FA2_ERR_INVALID_ARG;
    if (c->type != FA2_CACHE_SAME && c->type != FA2_CACHE_E4M3) return FA2_ERR_INVALID_ARG;
    if (dtype != FA2_DTYPE_F32 && dtype != FA2_DTYPE_F16 && dtype != FA2_DTYPE_BF16) return FA2_ERR_INVALID_ARG;
    const bool e4m3 = c->type == FA2_CACHE_E4M3;
    if (e4m3 && (!c->k_exp || !c->v_exp)) return FA2_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || c->n_kv_heads <= 0 || c->page_size <= 0 || c->head_dim <= 0 || batch <= 0 || pages_per_seq <= 0 ||
        table_stride < 0)
        return FA2_ERR_INVALID_ARG;
    if (batch > 1 && table_stride < pages_per_seq) return FA2_ERR_INVALID_ARG;
    const int64_t strides[3] = {c->page_stride, c->head_stride, c->slot_stride};
    const int64_t sizes[3] = {c->num_pages, c->n_kv_heads, c->page_size};
    if (!strides_ok(strides, 3) || !rows_apart(sizes, strides, 3, c->head_dim)) return FA2_ERR_INVALID_ARG;
    if (dtype == FA2_DTYPE_F32) return FA2_ERR_UNSUPPORTED;
    if (c->head_dim > 128 || c->head_dim % (e4m3 ? 16 : 8) != 0) return FA2_ERR_UNSUPPORTED;
    if (c->n_kv_heads > 1024 || c->num_pages > INT32_MAX || batch > kMaxGrid || c->page_size > kMaxLen ||
        pages_per_seq > kMaxLen || pages_per_seq * c->page_size > kMaxLen)
        return FA2_ERR_UNSUPPORTED;
    const int64_t eb = e4m3 ? 1 : 2;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(table, 4) || !aligned(lens, 4)) return FA2_ERR_MISALIGNED;
    for (int i = 0; i < 3; ++i)
        if (sizes[i] > 1 && strides[i] * eb % 16 != 0) return FA2_ERR_MISALIGNED;
    PagedParams& p = *out;
    p.k = static_cast<char*>(c->k); p.v = static_cast<char*>(c->v);
    p.k_exp = c->k_exp; p.v_exp = c->v_exp;
    p.num_pages = c->num_pages;
    p.page_stride = c->page_stride * eb; p.head_stride = c->head_stride * eb; p.slot_stride = c->slot_stride * eb;
    p.hkv = c->n_kv_heads; p.page_size = c->page_size; p.d = c->head_dim;
    page_divisor(p.page_size, &p.page_mul, &p.page_shift);
    p.e4m3 = e4m3;
    p.table = table; p.table_stride = table_stride; p.room = pages_per_seq * c->page_size;
    p.lens = lens; p.batch = batch; p.dtype = (int)dtype;
    return FA2_OK;
}

// The last step of every cache call: the watchdog word, then the launch.
template <typename Params>
fa2_status run(Params& p, cudaError_t (*launch)(const Params&, cudaStream_t), void* stream) {
    if (!watchdog_word(&p.c.status)) return FA2_ERR_CUDA;
    return launch(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA2_OK : FA2_ERR_CUDA;
}

}  // namespace

int32_t& decode_record() {
    thread_local int32_t record = -1;
    return record;
}

}  // namespace fa2

using namespace fa2;

extern "C" {

fa2_status fa2_rope_frequencies(double* inv_freq, float* magnitude, int32_t rot_dim, double base, fa2_rope_scaling scaling,
                                double factor, double original_len, double low, double high) {
    if (!inv_freq || rot_dim <= 0 || rot_dim % 2 != 0 || !(base > 0) || !isfinite(base)) return FA2_ERR_INVALID_ARG;
    if (scaling < FA2_ROPE_PLAIN || scaling > FA2_ROPE_RAMP) return FA2_ERR_INVALID_ARG;
    if (scaling != FA2_ROPE_PLAIN && (!(factor >= 1) || !isfinite(factor))) return FA2_ERR_INVALID_ARG;
    if (scaling == FA2_ROPE_BASE && rot_dim <= 2) return FA2_ERR_INVALID_ARG;
    const bool mixes = scaling == FA2_ROPE_TURNS || scaling == FA2_ROPE_RAMP;
    if (mixes && (!(original_len > 0) || !isfinite(original_len) || !(low > 0) || !(high > low) || !isfinite(high)))
        return FA2_ERR_INVALID_ARG;
    if (scaling == FA2_ROPE_RAMP && !(base > 1)) return FA2_ERR_INVALID_ARG;
    constexpr double kTwoPi = 6.283185307179586477;
    if (scaling == FA2_ROPE_BASE) base *= pow(factor, rot_dim / (rot_dim - 2.0));
    // the (fractional) index at which a frequency makes `turns` turns over the original length
    auto index_of = [&](double turns) { return rot_dim * log(original_len / (turns * kTwoPi)) / (2 * log(base)); };
    double from = 0, to = 0;
    if (scaling == FA2_ROPE_RAMP) {
        from = fmax(floor(index_of(high)), 0.0);
        to = fmin(ceil(index_of(low)), rot_dim - 1.0);
        if (!(to > from)) to = from + 0.001;  // a step
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot_dim);
        double w = 1;
        if (scaling == FA2_ROPE_LINEAR) w = 0;
        if (scaling == FA2_ROPE_TURNS) w = (original_len * f / kTwoPi - low) / (high - low);
        if (scaling == FA2_ROPE_RAMP) w = 1 - (i - from) / (to - from);
        w = fmin(fmax(w, 0.0), 1.0);
        inv_freq[i] = scaling == FA2_ROPE_PLAIN || scaling == FA2_ROPE_BASE ? f : f * (w + (1 - w) / factor);
    }
    if (magnitude) *magnitude = scaling == FA2_ROPE_RAMP ? (float)(0.1 * log(factor) + 1) : 1.f;
    return FA2_OK;
}

fa2_status fa2_rope(const void* x, void* y, const int32_t* positions, int64_t position_stride, const double* inv_freq,
                    int64_t b, int64_t h, int64_t n, int32_t head_dim, int32_t rot_dim, const int64_t x_strides[3],
                    const int64_t y_strides[3], int32_t interleaved, float magnitude, fa2_dtype dtype, void* stream) {
    return rope_call(x, y, positions, position_stride, inv_freq, b, h, n, head_dim, rot_dim, x_strides, y_strides,
                     interleaved, magnitude, dtype, stream, false);
}

fa2_status fa2_rope_backward(const void* dy, void* dx, const int32_t* positions, int64_t position_stride,
                             const double* inv_freq, int64_t b, int64_t h, int64_t n, int32_t head_dim, int32_t rot_dim,
                             const int64_t dy_strides[3], const int64_t dx_strides[3], int32_t interleaved,
                             float magnitude, fa2_dtype dtype, void* stream) {
    return rope_call(dy, dx, positions, position_stride, inv_freq, b, h, n, head_dim, rot_dim, dy_strides, dx_strides,
                     interleaved, magnitude, dtype, stream, true);
}

fa2_status fa2_kv_append(const fa2_kv_cache* cache, const void* k, const void* v, const int64_t k_strides[2],
                         const int64_t v_strides[2], const int32_t* block_table, int64_t table_stride,
                         int64_t pages_per_seq, const int32_t* cu_new, const int32_t* seq_lens, int64_t batch,
                         int64_t tokens, fa2_dtype dtype, void* stream) {
    if (!k || !v || !k_strides || !v_strides || tokens <= 0) return FA2_ERR_INVALID_ARG;
    if (!strides_ok(k_strides, 2) || !strides_ok(v_strides, 2)) return FA2_ERR_INVALID_ARG;
    if (!cu_new && tokens != batch) return FA2_ERR_INVALID_ARG;
    KvRowsParams p{};
    const fa2_status st = paged(cache, block_table, table_stride, pages_per_seq, seq_lens, batch, dtype, &p.c);
    if (st != FA2_OK) return st;
    if (tokens > INT32_MAX) return FA2_ERR_UNSUPPORTED;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_new, 4)) return FA2_ERR_MISALIGNED;
    const int64_t sizes[2] = {tokens, cache->n_kv_heads};
    for (int i = 0; i < 2; ++i)
        if (sizes[i] > 1 && (k_strides[i] % 8 != 0 || v_strides[i] % 8 != 0)) return FA2_ERR_MISALIGNED;
    p.k = static_cast<char*>(const_cast<void*>(k));
    p.v = static_cast<char*>(const_cast<void*>(v));
    for (int i = 0; i < 2; ++i) {
        p.ks[i] = k_strides[i] * 2;
        p.vs[i] = v_strides[i] * 2;
    }
    p.cu_new = cu_new;
    p.tokens = tokens;
    return run(p, launch_kv_rows, stream);
}

fa2_status fa2_kv_read(const fa2_kv_cache* cache, void* k_out, void* v_out, const int64_t out_strides[3],
                       const int32_t* block_table, int64_t table_stride, int64_t pages_per_seq,
                       const int32_t* seq_lens, int64_t batch, int64_t max_len, fa2_dtype dtype, void* stream) {
    if (!k_out || !v_out || !out_strides || max_len <= 0 || !strides_ok(out_strides, 3)) return FA2_ERR_INVALID_ARG;
    KvRowsParams p{};
    const fa2_status st = paged(cache, block_table, table_stride, pages_per_seq, seq_lens, batch, dtype, &p.c);
    if (st != FA2_OK) return st;
    if (max_len > kMaxLen) return FA2_ERR_UNSUPPORTED;
    const int64_t sizes[3] = {batch, cache->n_kv_heads, max_len};
    if (!rows_apart(sizes, out_strides, 3, cache->head_dim)) return FA2_ERR_INVALID_ARG;
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return FA2_ERR_MISALIGNED;
    for (int i = 0; i < 3; ++i)
        if (sizes[i] > 1 && out_strides[i] % 8 != 0) return FA2_ERR_MISALIGNED;
    p.k = static_cast<char*>(k_out);
    p.v = static_cast<char*>(v_out);
    for (int i = 0; i < 3; ++i) p.ks[i] = p.vs[i] = out_strides[i] * 2;
    p.tokens = max_len;
    p.read = true;
    return run(p, launch_kv_rows, stream);
}

size_t fa2_decode_workspace_size(int64_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
    if (batch <= 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 || head_dim <= 0 || head_dim > 128 ||
        head_dim % 8 != 0)
        return 0;
    return decode_workspace_bytes(n_heads, n_kv_heads, head_dim);
}

fa2_status fa2_decode(const void* q, const int64_t q_strides[2], const fa2_kv_cache* cache, void* o, float* lse,
                      const int32_t* block_table, int64_t table_stride, int64_t pages_per_seq,
                      const int32_t* seq_lens, int64_t batch, int32_t n_heads, int64_t window, void* workspace,
                      size_t workspace_bytes, fa2_dtype dtype, float softmax_scale, void* stream) {
    if (!q || !q_strides || !o || !lse || n_heads <= 0 || window < 0) return FA2_ERR_INVALID_ARG;
    if (!(softmax_scale > 0.f) || !isfinite(softmax_scale) || !strides_ok(q_strides, 2)) return FA2_ERR_INVALID_ARG;
    DecodeParams p{};
    const fa2_status st = paged(cache, block_table, table_stride, pages_per_seq, seq_lens, batch, dtype, &p.c);
    if (st != FA2_OK) return st;
    if (n_heads % cache->n_kv_heads != 0) return FA2_ERR_INVALID_ARG;
    if (n_heads > kMaxGrid || batch * n_heads > INT32_MAX) return FA2_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16)) return FA2_ERR_MISALIGNED;
    const int64_t sizes[2] = {batch, n_heads};
    for (int i = 0; i < 2; ++i)
        if (sizes[i] > 1 && q_strides[i] % 8 != 0) return FA2_ERR_MISALIGNED;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < decode_workspace_bytes(n_heads, cache->n_kv_heads, cache->head_dim))
        return FA2_ERR_WORKSPACE;
    p.q = q; p.q_batch = q_strides[0]; p.q_head = q_strides[1];
    p.o = o; p.lse = lse; p.heads = n_heads;
    p.window = window < p.c.room ? window : 0;  // as wide as the table: all keys
    p.workspace = static_cast<float*>(workspace);
    p.scale = softmax_scale;
    return run(p, launch_decode, stream);
}

fa2_status fa2_last_decode_info(int32_t* ctas_per_item) {
    if (!ctas_per_item) return FA2_ERR_INVALID_ARG;
    *ctas_per_item = decode_record();
    return FA2_OK;
}

}  // extern "C"
