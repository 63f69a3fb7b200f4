// layer_api.cpp -- the C ABI declared in include/kda_layer.h: argument
// validation on the host, then the launches on the caller's stream.
//
// Validation order as in kda_api.cpp: sizes, NULL pointers, supported
// configurations, alignment, aliasing (host checks only), then the device,
// then (debug mode) the offsets, then the launch.
#include "kda_api_common.h"
#include "kda_layer.h"
#include "layer_internal.h"

namespace {

bool aligned_to(const void *p, uint64_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

int elem_size(int32_t dtype) {
    return dtype == kda::kDtypeBf16 ? 2 : (dtype == kda::kDtypeF32 ? 4 : 0);
}

// The bytes of a tensor: `bytes` from the first to the last; with a stride, rows
// of `len` bytes that far apart (between them others' values may lie).
struct Span {
    const void *p;
    uint64_t bytes, stride, len;
    Span(const void *p_ = nullptr, uint64_t bytes_ = 0, uint64_t stride_ = 0, uint64_t len_ = 0)
        : p(p_), bytes(bytes_), stride(stride_), len(len_) {}
};
Span rows_range(const void *p, int64_t rows, int64_t len, int64_t stride, int esz) {
    if (rows <= 0 || len <= 0) return {p};
    return {p, (uint64_t)((rows - 1) * stride + len) * esz, (uint64_t)stride * esz,
            (uint64_t)len * esz};
}

// Rows the same distance apart whose columns lie beside each other (slices of
// one wider row) share no byte; everything else goes by first and last byte.
bool overlap(const Span &a, const Span &b) {
    if (!overlap(Range{a.p, a.bytes}, Range{b.p, b.bytes})) return false;
    if (a.stride == 0 || a.stride != b.stride) return true;
    const int64_t s = (int64_t)a.stride;
    const int64_t apart = (int64_t)reinterpret_cast<uintptr_t>(b.p) -
                          (int64_t)reinterpret_cast<uintptr_t>(a.p);
    const uint64_t d = (uint64_t)((apart % s + s) % s);  // b's column in a's row
    return d < a.len || d + b.len > a.stride;
}

// No output may overlap another output or an input.
template <int NO, int NI> int check_alias(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return KDA_ERR_ALIAS;
        for (int j = 0; j < NI; ++j)
            if (overlap(outs[i], ins[j])) return KDA_ERR_ALIAS;
    }
    return KDA_OK;
}

// Token numbers a little past the last one still fit 32 bits; a row of the
// convolution is addressed with 32-bit byte offsets.
constexpr int64_t kMostTokens = INT32_MAX - 4095;
constexpr int32_t kMostChannels = INT32_MAX / 4;

// Sizes of a call over sequences; *seqs receives them.
int check_seqs(const int32_t *cu, int32_t batch, int32_t seq_len, int32_t num_seqs,
               kda::Seqs *seqs) {
    if (batch < 0 || seq_len < 0) return KDA_ERR_SHAPE;
    if (cu && (batch != 1 || num_seqs < 0)) return KDA_ERR_SHAPE;
    const int64_t tokens = (int64_t)batch * seq_len;
    if (tokens > kMostTokens) return KDA_ERR_SHAPE;
    *seqs = {cu, cu ? num_seqs : batch, seq_len, (int32_t)tokens};
    return KDA_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------ short convolution
int kda_short_conv_fwd(const void *x, const float *weight, const float *bias,
                       const void *initial_state, const int32_t *cu_seqlens, void *out,
                       void *final_state, int32_t batch, int32_t seq_len, int32_t channels,
                       int32_t width, int64_t x_stride, int64_t out_stride, int32_t num_seqs,
                       int32_t activation, int32_t dtype, hipStream_t stream) {
    kda::Seqs seqs;
    int st = check_seqs(cu_seqlens, batch, seq_len, num_seqs, &seqs);
    if (st != KDA_OK) return st;
    if (channels < 0 || width < 1) return KDA_ERR_SHAPE;
    const int esz = elem_size(dtype);
    if (!esz) return KDA_ERR_UNSUPPORTED;
    const bool work = seqs.total > 0 && channels > 0;
    if (work && (x_stride < channels || out_stride < channels)) return KDA_ERR_SHAPE;
    if (work && (!x || !weight || !out)) return KDA_ERR_NULL;
    if (width < 2 || width > 4 || channels > kMostChannels) return KDA_ERR_UNSUPPORTED;
    if (activation != KDA_ACT_NONE && activation != KDA_ACT_SILU) return KDA_ERR_UNSUPPORTED;
    if (!aligned_to(x, esz) || !aligned_to(out, esz) || !aligned_to(initial_state, esz) ||
        !aligned_to(final_state, esz) || !aligned4(weight) || !aligned4(bias) ||
        !aligned4(cu_seqlens))
        return KDA_ERR_ALIGN;
    const uint64_t state = (uint64_t)seqs.num * (width - 1) * channels * esz;
    const Span outs[] = {rows_range(out, seqs.total, channels, out_stride, esz),
                          {final_state, state}};
    const Span ins[] = {rows_range(x, seqs.total, channels, x_stride, esz),
                         {weight, (uint64_t)channels * width * 4},
                         {bias, (uint64_t)channels * 4},
                         {initial_state, state},
                         {cu_seqlens, (uint64_t)(seqs.num + 1) * 4}};
    if ((st = check_alias(outs, ins)) != KDA_OK) return st;
    if (seqs.num == 0 || channels == 0) return KDA_OK;
    kda::ConvArgs a = {};
    a.x = x, a.state0 = initial_state, a.weight = weight, a.bias = bias, a.out = out;
    a.final_state = final_state, a.seqs = seqs, a.channels = channels, a.width = width;
    a.silu = activation == KDA_ACT_SILU, a.dtype = dtype;
    a.x_stride = x_stride, a.out_stride = out_stride;
    if (kda::conv_fwd_threads(a) > kda::kMostThreads) return KDA_ERR_UNSUPPORTED;
    if ((st = check_device()) != KDA_OK) return st;
    const char *where = "kda_short_conv_fwd";
    if (debug_mode() &&
        (st = debug_check_offsets(cu_seqlens, seqs.num, seqs.total, stream, where)) != KDA_OK)
        return st;
    return launch_status(kda::launch_conv_fwd(a, stream), stream, where);
}

int64_t kda_short_conv_bwd_workspace_size(int32_t batch, int32_t seq_len, int32_t channels,
                                          int32_t width) {
    if (batch < 0 || seq_len < 0 || channels < 0 || width < 2 || width > 4) return -1;
    const int64_t tokens = (int64_t)batch * seq_len;
    if (tokens > kMostTokens || channels > kMostChannels) return -1;
    return 4 * kda::conv_bwd_workspace_floats(tokens, channels, width);
}

int kda_short_conv_bwd(const void *x, const float *weight, const float *bias,
                       const void *initial_state, const int32_t *cu_seqlens, const void *d_out,
                       const void *d_final_state, void *dx, float *dweight, float *dbias,
                       void *d_initial_state, int32_t batch, int32_t seq_len, int32_t channels,
                       int32_t width, int64_t x_stride, int64_t d_out_stride, int64_t dx_stride,
                       int32_t num_seqs, int32_t activation, int32_t dtype, void *workspace,
                       int64_t workspace_bytes, hipStream_t stream) {
    kda::Seqs seqs;
    int st = check_seqs(cu_seqlens, batch, seq_len, num_seqs, &seqs);
    if (st != KDA_OK) return st;
    if (channels < 0 || width < 1) return KDA_ERR_SHAPE;
    const int esz = elem_size(dtype);
    if (!esz) return KDA_ERR_UNSUPPORTED;
    const bool work = seqs.total > 0 && channels > 0;
    if (work && (x_stride < channels || d_out_stride < channels || dx_stride < channels))
        return KDA_ERR_SHAPE;
    if (work && (!x || !d_out || !dx)) return KDA_ERR_NULL;
    if (channels > 0 && (!weight || !dweight)) return KDA_ERR_NULL;
    if (width < 2 || width > 4 || channels > kMostChannels) return KDA_ERR_UNSUPPORTED;
    if (activation != KDA_ACT_NONE && activation != KDA_ACT_SILU) return KDA_ERR_UNSUPPORTED;
    const int64_t need = 4 * kda::conv_bwd_workspace_floats(seqs.total, channels, width);
    if (need > 0 && !workspace) return KDA_ERR_NULL;
    if (workspace_bytes < need) return KDA_ERR_SHAPE;
    if (!aligned_to(x, esz) || !aligned_to(d_out, esz) || !aligned_to(dx, esz) ||
        !aligned_to(initial_state, esz) || !aligned_to(d_final_state, esz) ||
        !aligned_to(d_initial_state, esz) || !aligned4(weight) || !aligned4(bias) ||
        !aligned4(dweight) || !aligned4(dbias) || !aligned4(cu_seqlens) || !aligned16(workspace))
        return KDA_ERR_ALIGN;
    const uint64_t state = (uint64_t)seqs.num * (width - 1) * channels * esz;
    const uint64_t wb = (uint64_t)channels * width * 4, bb = (uint64_t)channels * 4;
    const Span outs[] = {rows_range(dx, seqs.total, channels, dx_stride, esz),
                          {dweight, wb},
                          {dbias, bb},
                          {d_initial_state, state},
                          {workspace, (uint64_t)need}};
    const Span ins[] = {rows_range(x, seqs.total, channels, x_stride, esz),
                         rows_range(d_out, seqs.total, channels, d_out_stride, esz),
                         {weight, wb},
                         {bias, bb},
                         {initial_state, state},
                         {d_final_state, state},
                         {cu_seqlens, (uint64_t)(seqs.num + 1) * 4}};
    if ((st = check_alias(outs, ins)) != KDA_OK) return st;
    if (channels == 0) return KDA_OK;
    const int32_t tokens = seqs.total;
    if (seqs.num == 0) seqs.total = 0;  // no sequence holds a token
    kda::ConvArgs a = {};
    a.x = x, a.state0 = initial_state, a.d_out = d_out, a.d_final = d_final_state;
    a.weight = weight, a.bias = bias, a.dx = dx, a.d_state0 = d_initial_state;
    a.dweight = dweight, a.dbias = dbias, a.partial = static_cast<float *>(workspace);
    a.seqs = seqs, a.channels = channels, a.width = width;
    a.silu = activation == KDA_ACT_SILU, a.dtype = dtype;
    a.x_stride = x_stride, a.d_out_stride = d_out_stride, a.dx_stride = dx_stride;
    if (kda::conv_bwd_threads(a) > kda::kMostThreads) return KDA_ERR_UNSUPPORTED;
    if ((st = check_device()) != KDA_OK) return st;
    const char *where = "kda_short_conv_bwd";
    if (debug_mode() &&
        (st = debug_check_offsets(cu_seqlens, seqs.num, tokens, stream, where)) != KDA_OK)
        return st;
    return launch_status(kda::launch_conv_bwd(a, stream), stream, where);
}

int kda_short_conv_step(const void *x, const float *weight, const float *bias, void *state,
                        void *out, int32_t batch, int32_t channels, int32_t width,
                        int64_t x_stride, int64_t out_stride, int32_t activation, int32_t dtype,
                        hipStream_t stream) {
    if (batch < 0 || channels < 0 || width < 1) return KDA_ERR_SHAPE;
    const int esz = elem_size(dtype);
    if (!esz) return KDA_ERR_UNSUPPORTED;
    const bool work = batch > 0 && channels > 0;
    if (work && (x_stride < channels || out_stride < channels)) return KDA_ERR_SHAPE;
    if (work && (!x || !weight || !state || !out)) return KDA_ERR_NULL;
    if (width < 2 || width > 4 || channels > kMostChannels) return KDA_ERR_UNSUPPORTED;
    if (activation != KDA_ACT_NONE && activation != KDA_ACT_SILU) return KDA_ERR_UNSUPPORTED;
    if (!aligned_to(x, esz) || !aligned_to(out, esz) || !aligned_to(state, esz) ||
        !aligned4(weight) || !aligned4(bias))
        return KDA_ERR_ALIGN;
    const Span outs[] = {rows_range(out, batch, channels, out_stride, esz),
                          {state, (uint64_t)batch * (width - 1) * channels * esz}};
    const Span ins[] = {rows_range(x, batch, channels, x_stride, esz),
                         {weight, (uint64_t)channels * width * 4},
                         {bias, (uint64_t)channels * 4}};
    int st = check_alias(outs, ins);
    if (st != KDA_OK) return st;
    if (!work) return KDA_OK;
    kda::ConvArgs a = {};
    a.x = x, a.weight = weight, a.bias = bias, a.out = out;
    a.channels = channels, a.width = width, a.silu = activation == KDA_ACT_SILU, a.dtype = dtype;
    a.x_stride = x_stride, a.out_stride = out_stride;
    if (kda::conv_step_threads(a, state, batch) > kda::kMostThreads) return KDA_ERR_UNSUPPORTED;
    if ((st = check_device()) != KDA_OK) return st;
    return launch_status(kda::launch_conv_step(a, state, batch, stream), stream,
                         "kda_short_conv_step");
}

}  // extern "C"

// ------------------------------------------------------------ norm and rotation
namespace {

// Checks shared by both directions; the spans of q, k, weights, table and
// positions go to `ins` (six of them).
int check_qk(const void *q, const void *k, const float *q_weight, const float *k_weight,
             const float *table, const int32_t *positions, int32_t tokens, int32_t q_heads,
             int32_t k_heads, int32_t head_dim, int32_t rotary_dim, int32_t table_rows,
             int64_t q_stride, int64_t k_stride, float eps, int32_t norm, int32_t dtype,
             Span (&ins)[6]) {
    if (tokens < 0 || q_heads < 0 || k_heads < 0 || head_dim <= 0 || rotary_dim < 0)
        return KDA_ERR_SHAPE;
    // the kernels address a token's heads with 32-bit byte offsets
    if (((int64_t)q_heads + k_heads) * head_dim > INT32_MAX / 4) return KDA_ERR_UNSUPPORTED;
    if (rotary_dim > head_dim || !(eps >= 0.f)) return KDA_ERR_SHAPE;
    const int esz = elem_size(dtype);
    if (!esz) return KDA_ERR_UNSUPPORTED;
    const int64_t ql = (int64_t)q_heads * head_dim, kl = (int64_t)k_heads * head_dim;
    const bool any_q = tokens > 0 && q_heads > 0, any_k = tokens > 0 && k_heads > 0;
    if ((any_q && q_stride < ql) || (any_k && k_stride < kl)) return KDA_ERR_SHAPE;
    if ((any_q && !q) || (any_k && !k)) return KDA_ERR_NULL;
    if (rotary_dim > 0 && (any_q || any_k)) {
        if (!table || !positions) return KDA_ERR_NULL;
        if (table_rows < 1) return KDA_ERR_SHAPE;
    }
    if (head_dim != 64 && head_dim != 128) return KDA_ERR_UNSUPPORTED;
    if (rotary_dim % 16 != 0) return KDA_ERR_UNSUPPORTED;
    if (norm != KDA_NORM_L2 && norm != KDA_NORM_RMS) return KDA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(table) || !aligned4(positions) ||
        !aligned4(q_weight) || !aligned4(k_weight) || (any_q && q_stride * esz % 16 != 0) ||
        (any_k && k_stride * esz % 16 != 0))
        return KDA_ERR_ALIGN;
    const bool rot = rotary_dim > 0;
    ins[0] = rows_range(q, tokens, ql, q_stride, esz);
    ins[1] = rows_range(k, tokens, kl, k_stride, esz);
    ins[2] = {q_weight, (uint64_t)head_dim * 4};
    ins[3] = {k_weight, (uint64_t)head_dim * 4};
    ins[4] = {rot ? table : nullptr, rot ? (uint64_t)table_rows * rotary_dim * 4 : 0};
    ins[5] = {rot ? positions : nullptr, (uint64_t)tokens * 4};
    return KDA_OK;
}

// One more pair of tensors laid out like q and k.
int check_qk_rows(const void *q, const void *k, int32_t tokens, int32_t q_heads, int32_t k_heads,
                  int32_t head_dim, int64_t q_stride, int64_t k_stride, int32_t dtype, Span *r) {
    const int esz = elem_size(dtype);
    const int64_t ql = (int64_t)q_heads * head_dim, kl = (int64_t)k_heads * head_dim;
    const bool any_q = tokens > 0 && q_heads > 0, any_k = tokens > 0 && k_heads > 0;
    if ((any_q && q_stride < ql) || (any_k && k_stride < kl)) return KDA_ERR_SHAPE;
    if ((any_q && !q) || (any_k && !k)) return KDA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || (any_q && q_stride * esz % 16 != 0) ||
        (any_k && k_stride * esz % 16 != 0))
        return KDA_ERR_ALIGN;
    r[0] = rows_range(q, tokens, ql, q_stride, esz);
    r[1] = rows_range(k, tokens, kl, k_stride, esz);
    return KDA_OK;
}

}  // namespace

extern "C" {

int kda_qk_norm_fwd(const void *q, const void *k, const float *q_weight, const float *k_weight,
                    const float *table, const int32_t *positions, void *out_q, void *out_k,
                    int32_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                    int32_t rotary_dim, int32_t table_rows, int64_t q_stride, int64_t k_stride,
                    int64_t out_q_stride, int64_t out_k_stride, float eps, int32_t norm,
                    int32_t interleaved, int32_t dtype, hipStream_t stream) {
    Span ins[6], outs[2];
    int st = check_qk(q, k, q_weight, k_weight, table, positions, tokens, q_heads, k_heads,
                      head_dim, rotary_dim, table_rows, q_stride, k_stride, eps, norm, dtype, ins);
    if (st != KDA_OK) return st;
    st = check_qk_rows(out_q, out_k, tokens, q_heads, k_heads, head_dim, out_q_stride,
                       out_k_stride, dtype, outs);
    if (st != KDA_OK) return st;
    if ((st = check_alias(outs, ins)) != KDA_OK) return st;
    if (tokens == 0 || (q_heads == 0 && k_heads == 0)) return KDA_OK;
    if ((st = check_device()) != KDA_OK) return st;
    const kda::QkArgs a = {{q, k},       {nullptr, nullptr}, {out_q, out_k},
                           {q_weight, k_weight}, {nullptr, nullptr}, nullptr,
                           table,        positions,          tokens,
                           {q_heads, k_heads}, head_dim,     rotary_dim,
                           table_rows,   {q_stride, k_stride}, {0, 0},
                           {out_q_stride, out_k_stride}, eps, norm == KDA_NORM_RMS,
                           interleaved != 0, dtype};
    return launch_status(kda::launch_qk_norm_fwd(a, stream), stream, "kda_qk_norm_fwd");
}

int64_t kda_qk_norm_bwd_workspace_size(int32_t tokens, int32_t q_heads, int32_t k_heads,
                                       int32_t head_dim) {
    if (tokens < 0 || q_heads < 0 || k_heads < 0 || (head_dim != 64 && head_dim != 128) ||
        ((int64_t)q_heads + k_heads) * head_dim > INT32_MAX / 4)
        return -1;
    return 4 * kda::qk_norm_bwd_workspace_floats(tokens, q_heads, k_heads, head_dim);
}

int kda_qk_norm_bwd(const void *q, const void *k, const float *q_weight, const float *k_weight,
                    const float *table, const int32_t *positions, const void *d_out_q,
                    const void *d_out_k, void *dq, void *dk, float *dq_weight, float *dk_weight,
                    int32_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                    int32_t rotary_dim, int32_t table_rows, int64_t q_stride, int64_t k_stride,
                    int64_t d_out_q_stride, int64_t d_out_k_stride, int64_t dq_stride,
                    int64_t dk_stride, float eps, int32_t norm, int32_t interleaved,
                    int32_t dtype, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    Span ins[8], outs[5], base[6];
    int st = check_qk(q, k, q_weight, k_weight, table, positions, tokens, q_heads, k_heads,
                      head_dim, rotary_dim, table_rows, q_stride, k_stride, eps, norm, dtype,
                      base);
    if (st != KDA_OK) return st;
    // the gradient of a weight that was not given has no meaning
    if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return KDA_ERR_NULL;
    for (int i = 0; i < 6; ++i) ins[i] = base[i];
    st = check_qk_rows(d_out_q, d_out_k, tokens, q_heads, k_heads, head_dim, d_out_q_stride,
                       d_out_k_stride, dtype, ins + 6);
    if (st != KDA_OK) return st;
    st = check_qk_rows(dq, dk, tokens, q_heads, k_heads, head_dim, dq_stride, dk_stride, dtype,
                       outs);
    if (st != KDA_OK) return st;
    const bool weights = dq_weight || dk_weight;
    const int64_t need =
        weights ? kda_qk_norm_bwd_workspace_size(tokens, q_heads, k_heads, head_dim) : 0;
    if (need > 0 && !workspace) return KDA_ERR_NULL;
    if (workspace_bytes < need) return KDA_ERR_SHAPE;
    if (!aligned4(dq_weight) || !aligned4(dk_weight) || !aligned16(workspace))
        return KDA_ERR_ALIGN;
    outs[2] = {dq_weight, (uint64_t)head_dim * 4};
    outs[3] = {dk_weight, (uint64_t)head_dim * 4};
    outs[4] = {workspace, (uint64_t)need};
    if ((st = check_alias(outs, ins)) != KDA_OK) return st;
    const bool none = tokens == 0 || (q_heads == 0 && k_heads == 0);
    if (none && !weights) return KDA_OK;
    if ((st = check_device()) != KDA_OK) return st;
    kda::QkArgs a = {{q, k},       {d_out_q, d_out_k}, {dq, dk},
                     {q_weight, k_weight}, {dq_weight, dk_weight}, static_cast<float *>(workspace),
                     table,        positions,          none ? 0 : tokens,
                     {q_heads, k_heads}, head_dim,     rotary_dim,
                     table_rows,   {q_stride, k_stride}, {d_out_q_stride, d_out_k_stride},
                     {dq_stride, dk_stride}, eps,      norm == KDA_NORM_RMS,
                     interleaved != 0, dtype};
    return launch_status(kda::launch_qk_norm_bwd(a, stream), stream, "kda_qk_norm_bwd");
}

}  // extern "C"

// ------------------------------------------------------------ state space scan
namespace {

// Sizes and supported configurations of the scan.
int check_ssm_dims(int32_t heads, int32_t groups, int32_t p, int32_t n, int32_t dtype) {
    if (heads < 0 || groups < 0 || p <= 0 || n <= 0) return KDA_ERR_SHAPE;
    if (heads > 0 && (groups == 0 || heads % groups != 0)) return KDA_ERR_SHAPE;
    if (!elem_size(dtype)) return KDA_ERR_UNSUPPORTED;
    if ((p != 64 && p != 128) || (n != 64 && n != 128)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// A tensor of `rows` token rows of `len` elements: stride and alignment.
int check_ssm_rows(const void *t, int64_t rows, int64_t len, int64_t stride, int esz) {
    if (rows > 0 && len > 0) {
        if (stride < len) return KDA_ERR_SHAPE;
        if (!t) return KDA_ERR_NULL;
        // the kernels address 64 rows with 32-bit byte offsets
        if (stride > INT32_MAX / (64 * esz)) return KDA_ERR_UNSUPPORTED;
        if (stride * esz % 16 != 0) return KDA_ERR_ALIGN;
    }
    return aligned16(t) ? KDA_OK : KDA_ERR_ALIGN;
}

// How a call's sequences are cut (host rule, from sizes alone): pieces of
// `len` tokens, or one piece per sequence (split = false).
struct PiecePlan {
    bool split;
    int32_t len;
};
PiecePlan piece_plan(const kda::Seqs &s, int32_t heads, int32_t p, int directions) {
    // 512 workgroups of 128 state rows, two a CU, in one round (both directions of
    // the backward are one launch).  Measured with two bf16 parts where y, dB and dC
    // take three now: 32K x 64 heads of 64 rows 384 us, with 256 workgroups 477, with
    // 1024 409; of 128 rows 690, with 1024 723.  8K backward 549 us, with 256 613, with
    // 1024 567.  Equal rows that come to half of that are left whole.
    const int64_t want = 512 / directions, units = ((int64_t)heads * p + 127) / 128;
    const bool enough = !s.cu && s.num * units >= want / 2;
    // Down to one block of 64 tokens (1,227 tokens x 8 heads fp32: 30 us, against
    // 47 us with 256), but at most 64 pieces a sequence: the fold walks them.
    const int64_t longest = s.cu ? s.total : s.seq_len;
    int64_t len = (s.total * units + want - 1) / want;
    if (len < longest / 64) len = longest / 64;
    len = (len + 63) / 64 * 64;
    if (len < 64) len = 64;
    if (len > (1 << 20)) len = 1 << 20;
    if (enough || longest <= len) {
        int64_t whole = (longest + 63) / 64 * 64;
        return {false, (int32_t)(whole < 64 ? 64 : (whole > INT32_MAX - 63 ? INT32_MAX - 63 : whole))};
    }
    return {true, (int32_t)len};
}
struct SsmSpace {
    int64_t states, decay;  // floats of the piece states, doubles of their decays
    int64_t bytes() const { return 8 * ((decay + 1) / 2 * 2) + 4 * states; }
};
SsmSpace ssm_space(const kda::Seqs &s, int32_t heads, int32_t p, int32_t n, int directions = 1) {
    const PiecePlan plan = piece_plan(s, heads, p, directions);
    if (!plan.split || s.num == 0) return {0, 0};
    const int64_t count = kda::slot_count(s, plan.len) * heads;
    return {count * p * n, count};
}

}  // namespace

extern "C" {

int64_t kda_ssm_chunk_fwd_workspace_size(int32_t batch, int32_t seq_len, int32_t num_seqs,
                                         int32_t num_heads, int32_t head_dim, int32_t state_dim) {
    static const int32_t packed = 0;  // stands for offsets; never read
    kda::Seqs seqs;
    if (check_seqs(num_seqs > 0 ? &packed : nullptr, batch, seq_len, num_seqs, &seqs) != KDA_OK ||
        check_ssm_dims(num_heads, 1, head_dim, state_dim, kda::kDtypeF32) != KDA_OK)
        return -1;
    return ssm_space(seqs, num_heads, head_dim, state_dim).bytes();
}

int kda_ssm_chunk_fwd(const void *x, const float *dt, const float *A, const void *B,
                      const void *C, const float *D, const float *initial_state,
                      const int32_t *cu_seqlens, void *out, float *final_state, int32_t batch,
                      int32_t seq_len, int32_t num_heads, int32_t num_groups, int32_t head_dim,
                      int32_t state_dim, int64_t x_stride, int64_t b_stride, int64_t c_stride,
                      int64_t out_stride, int32_t num_seqs, int32_t dtype, void *workspace,
                      int64_t workspace_bytes, hipStream_t stream) {
    kda::Seqs seqs;
    int st = check_seqs(cu_seqlens, batch, seq_len, num_seqs, &seqs);
    if (st != KDA_OK) return st;
    if ((st = check_ssm_dims(num_heads, num_groups, head_dim, state_dim, dtype)) != KDA_OK)
        return st;
    const int esz = elem_size(dtype);
    const int64_t xl = (int64_t)num_heads * head_dim;
    const int64_t bl = num_heads > 0 ? (int64_t)num_groups * state_dim : 0;
    const int64_t th = (int64_t)seqs.total * num_heads;
    if (th > 0 && !dt) return KDA_ERR_NULL;
    if (seqs.num > 0 && num_heads > 0 && !A) return KDA_ERR_NULL;  // read without tokens too
    if ((st = check_ssm_rows(x, seqs.total, xl, x_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(B, seqs.total, bl, b_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(C, seqs.total, bl, c_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(out, seqs.total, xl, out_stride, esz)) != KDA_OK)
        return st;
    const SsmSpace space = ssm_space(seqs, num_heads, head_dim, state_dim);
    if (space.bytes() > 0 && !workspace) return KDA_ERR_NULL;
    if (workspace_bytes < space.bytes()) return KDA_ERR_SHAPE;
    if (!aligned4(dt) || !aligned4(A) || !aligned4(D) || !aligned16(initial_state) ||
        !aligned16(final_state) || !aligned4(cu_seqlens) || !aligned16(workspace))
        return KDA_ERR_ALIGN;
    const uint64_t state = (uint64_t)seqs.num * xl * state_dim * 4;
    const Span outs[] = {rows_range(out, seqs.total, xl, out_stride, esz),
                          {workspace, (uint64_t)space.bytes()},
                          {final_state, state}};
    const Span ins[] = {rows_range(x, seqs.total, xl, x_stride, esz),
                         rows_range(B, seqs.total, bl, b_stride, esz),
                         rows_range(C, seqs.total, bl, c_stride, esz),
                         {dt, (uint64_t)th * 4},
                         {A, (uint64_t)num_heads * 4},
                         {D, (uint64_t)num_heads * 4},
                         {cu_seqlens, (uint64_t)(seqs.num + 1) * 4},
                         {final_state == initial_state ? nullptr : initial_state, state}};
    if ((st = check_alias(outs, ins)) != KDA_OK) return st;
    if (final_state == initial_state &&  // in place: still apart from the other outputs
        (overlap(outs[0], Span{initial_state, state}) || overlap(outs[1], Span{initial_state, state})))
        return KDA_ERR_ALIAS;
    if (seqs.num == 0 || num_heads == 0) return KDA_OK;
    kda::SsmScan a = {};
    a.x = x, a.k = B, a.c = C, a.dt = dt, a.A = A, a.D = D, a.state0 = initial_state;
    a.out = out, a.final_state = final_state, a.seqs = seqs;
    a.heads = num_heads, a.groups = num_groups, a.p = head_dim, a.n = state_dim;
    a.piece = piece_plan(seqs, num_heads, head_dim, 1).len;
    a.x_stride = x_stride, a.k_stride = b_stride, a.c_stride = c_stride;
    a.out_stride = out_stride;
    if (space.states > 0) {
        a.seg_decay = static_cast<double *>(workspace);
        a.seg_states = reinterpret_cast<float *>(a.seg_decay + (space.decay + 1) / 2 * 2);
    }
    if (kda::ssm_scan_threads(a, dtype, 1) > kda::kMostThreads) return KDA_ERR_UNSUPPORTED;
    if ((st = check_device()) != KDA_OK) return st;
    const char *where = "kda_ssm_chunk_fwd";
    if (debug_mode() &&
        (st = debug_check_offsets(cu_seqlens, seqs.num, seqs.total, stream, where)) != KDA_OK)
        return st;
    return launch_status(kda::launch_ssm_out(a, dtype, stream), stream, where);
}

}  // extern "C"

namespace {

// The backward's workspace: piece decays and states (the forward's, twice), the
// states at every block from both sides, the parts of dA and dD, and with
// several sets of heads the parts of dB and dC.
struct SsmBwdSpace {
    SsmSpace pieces;
    int64_t blocks, states, params, bc;  // block numbers; floats of each part
    int32_t sets;
    int64_t bytes() const { return 2 * pieces.bytes() + 4 * (2 * states + params + bc); }
};
SsmBwdSpace ssm_bwd_space(const kda::Seqs &s, int32_t heads, int32_t groups, int32_t p, int32_t n,
                          int32_t dtype) {
    SsmBwdSpace w = {};
    if (s.num == 0 || heads == 0) return w;
    w.pieces = ssm_space(s, heads, p, n, 2);
    const int64_t block = dtype == kda::kDtypeBf16 ? 64 : 32;
    w.blocks = kda::piece_count(s, block);
    w.states = w.blocks * heads * p * n;
    w.params = (2 * w.blocks * heads + 3) / 4 * 4;
    // sets: enough workgroups to fill the chip twice over
    const int64_t units = w.blocks * groups, per_group = heads / groups;
    int64_t sets = (512 + units - 1) / units;
    sets = sets > per_group ? per_group : sets;
    const int64_t per_set = (per_group + sets - 1) / sets;
    w.sets = (int32_t)((per_group + per_set - 1) / per_set);
    w.bc = w.sets > 1 ? 2 * w.sets * (int64_t)s.total * groups * n : 0;
    return w;
}

}  // namespace

extern "C" {

int64_t kda_ssm_chunk_bwd_workspace_size(int32_t batch, int32_t seq_len, int32_t num_seqs,
                                         int32_t num_heads, int32_t num_groups, int32_t head_dim,
                                         int32_t state_dim, int32_t dtype) {
    static const int32_t packed = 0;  // stands for offsets; never read
    kda::Seqs seqs;
    if (check_seqs(num_seqs > 0 ? &packed : nullptr, batch, seq_len, num_seqs, &seqs) != KDA_OK ||
        check_ssm_dims(num_heads, num_groups, head_dim, state_dim, dtype) != KDA_OK)
        return -1;
    return ssm_bwd_space(seqs, num_heads, num_groups, head_dim, state_dim, dtype).bytes();
}

int kda_ssm_chunk_bwd(const void *x, const float *dt, const float *A, const void *B,
                      const void *C, const float *D, const float *initial_state,
                      const int32_t *cu_seqlens, const void *d_out, const float *d_final_state,
                      void *dx, float *ddt, float *dA, void *dB, void *dC, float *dD,
                      float *d_initial_state, int32_t batch, int32_t seq_len, int32_t num_heads,
                      int32_t num_groups, int32_t head_dim, int32_t state_dim, int64_t x_stride,
                      int64_t b_stride, int64_t c_stride, int64_t d_out_stride,
                      int64_t dx_stride, int64_t db_stride, int64_t dc_stride, int32_t num_seqs,
                      int32_t dtype, void *workspace, int64_t workspace_bytes,
                      hipStream_t stream) {
    kda::Seqs seqs;
    int st = check_seqs(cu_seqlens, batch, seq_len, num_seqs, &seqs);
    if (st != KDA_OK) return st;
    if ((st = check_ssm_dims(num_heads, num_groups, head_dim, state_dim, dtype)) != KDA_OK)
        return st;
    const int esz = elem_size(dtype);
    const int64_t xl = (int64_t)num_heads * head_dim;
    const int64_t bl = num_heads > 0 ? (int64_t)num_groups * state_dim : 0;
    const int64_t th = (int64_t)seqs.total * num_heads;
    if (th > 0 && (!dt || !ddt)) return KDA_ERR_NULL;
    if (num_heads > 0 && (!A || !dA)) return KDA_ERR_NULL;
    if (dD && !D) return KDA_ERR_NULL;  // the gradient of what was not given
    if ((st = check_ssm_rows(x, seqs.total, xl, x_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(B, seqs.total, bl, b_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(C, seqs.total, bl, c_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(d_out, seqs.total, xl, d_out_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(dx, seqs.total, xl, dx_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(dB, seqs.total, bl, db_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(dC, seqs.total, bl, dc_stride, esz)) != KDA_OK)
        return st;
    const SsmBwdSpace w =
        ssm_bwd_space(seqs, num_heads, num_groups, head_dim, state_dim, dtype);
    if (w.bytes() > 0 && !workspace) return KDA_ERR_NULL;
    if (workspace_bytes < w.bytes()) return KDA_ERR_SHAPE;
    if (!aligned4(dt) || !aligned4(A) || !aligned4(D) || !aligned16(initial_state) ||
        !aligned16(d_final_state) || !aligned16(d_initial_state) || !aligned4(cu_seqlens) ||
        !aligned4(ddt) || !aligned4(dA) || !aligned4(dD) || !aligned16(workspace))
        return KDA_ERR_ALIGN;
    const uint64_t state = (uint64_t)seqs.num * xl * state_dim * 4, hb = (uint64_t)num_heads * 4;
    const Span outs[] = {rows_range(dx, seqs.total, xl, dx_stride, esz),
                          rows_range(dB, seqs.total, bl, db_stride, esz),
                          rows_range(dC, seqs.total, bl, dc_stride, esz),
                          {ddt, (uint64_t)th * 4},
                          {dA, hb},
                          {dD, hb},
                          {d_initial_state, state},
                          {workspace, (uint64_t)w.bytes()}};
    const Span ins[] = {rows_range(x, seqs.total, xl, x_stride, esz),
                         rows_range(B, seqs.total, bl, b_stride, esz),
                         rows_range(C, seqs.total, bl, c_stride, esz),
                         rows_range(d_out, seqs.total, xl, d_out_stride, esz),
                         {dt, (uint64_t)th * 4},
                         {A, hb},
                         {D, hb},
                         {cu_seqlens, (uint64_t)(seqs.num + 1) * 4},
                         {initial_state, state},
                         {d_final_state, state}};
    if ((st = check_alias(outs, ins)) != KDA_OK) return st;
    if (num_heads == 0) return KDA_OK;
    kda::SsmGrad g = {};
    g.dA = dA, g.dD = dD, g.seqs = seqs, g.heads = num_heads, g.groups = num_groups;
    kda::SsmScan a = {}, b = {};  // from the left, from the right
    if (seqs.num > 0) {
        a.x = x, a.k = B, a.dt = dt, a.A = A, a.state0 = initial_state;
        a.seqs = seqs, a.heads = num_heads, a.groups = num_groups;
        a.p = head_dim, a.n = state_dim, a.piece = piece_plan(seqs, num_heads, head_dim, 2).len;
        a.x_stride = x_stride, a.k_stride = b_stride;
        b = a;
        b.x = d_out, b.k = C, b.x_stride = d_out_stride, b.k_stride = c_stride;
        b.state0 = d_final_state, b.final_state = d_initial_state;
        char *at = static_cast<char *>(workspace);
        if (w.pieces.states > 0) {
            const int64_t decays = (w.pieces.decay + 1) / 2 * 2;
            a.seg_decay = reinterpret_cast<double *>(at);
            b.seg_decay = a.seg_decay + decays;
            a.seg_states = reinterpret_cast<float *>(b.seg_decay + decays);
            b.seg_states = a.seg_states + w.pieces.states;
        }
        a.block_states = reinterpret_cast<float *>(at + 2 * w.pieces.bytes());
        b.block_states = a.block_states + w.states;
        g.x = x, g.B = B, g.C = C, g.dy = d_out, g.dt = dt, g.A = A, g.D = D;
        g.s_states = a.block_states, g.e_states = b.block_states;
        g.dx = dx, g.dB = dB, g.dC = dC, g.ddt = ddt;
        g.part_a = b.block_states + w.states, g.part_d = g.part_a + w.blocks * num_heads;
        g.part_bc = g.part_a + w.params;
        g.p = head_dim, g.n = state_dim, g.sets = w.sets, g.blocks = w.blocks;
        g.x_stride = x_stride, g.b_stride = b_stride, g.c_stride = c_stride;
        g.dy_stride = d_out_stride, g.dx_stride = dx_stride;
        g.db_stride = db_stride, g.dc_stride = dc_stride;
        if (kda::ssm_scan_threads(a, dtype, 2) > kda::kMostThreads ||
            kda::ssm_grad_threads(g) > kda::kMostThreads)
            return KDA_ERR_UNSUPPORTED;
    }
    if ((st = check_device()) != KDA_OK) return st;
    const char *where = "kda_ssm_chunk_bwd";
    if (debug_mode() &&
        (st = debug_check_offsets(cu_seqlens, seqs.num, seqs.total, stream, where)) != KDA_OK)
        return st;
    if (seqs.num > 0) {
        const int rc = kda::launch_ssm_states(a, b, dtype, stream);
        if (rc != 0) return launch_status(rc, stream, where);
    }
    return launch_status(kda::launch_ssm_grad(g, dtype, stream), stream, where);
}

int kda_ssm_decode_step(const void *x, const float *dt, const float *A, const void *B,
                        const void *C, const float *D, float *state, void *out, int32_t batch,
                        int32_t num_heads, int32_t num_groups, int32_t head_dim,
                        int32_t state_dim, int64_t x_stride, int64_t b_stride, int64_t c_stride,
                        int64_t out_stride, int32_t dtype, hipStream_t stream) {
    if (batch < 0) return KDA_ERR_SHAPE;
    int st = check_ssm_dims(num_heads, num_groups, head_dim, state_dim, dtype);
    if (st != KDA_OK) return st;
    const int esz = elem_size(dtype);
    const int64_t xl = (int64_t)num_heads * head_dim;
    const int64_t bl = num_heads > 0 ? (int64_t)num_groups * state_dim : 0;
    const uint64_t units = (uint64_t)batch * num_heads;
    if (units * kda::kSsmStepThreads > (uint64_t)kda::kMostThreads) return KDA_ERR_UNSUPPORTED;
    if (units > 0 && (!dt || !A || !state)) return KDA_ERR_NULL;
    if ((st = check_ssm_rows(x, batch, xl, x_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(B, batch, bl, b_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(C, batch, bl, c_stride, esz)) != KDA_OK ||
        (st = check_ssm_rows(out, batch, xl, out_stride, esz)) != KDA_OK)
        return st;
    if (!aligned4(dt) || !aligned4(A) || !aligned4(D) || !aligned16(state)) return KDA_ERR_ALIGN;
    const Span outs[] = {rows_range(out, batch, xl, out_stride, esz),
                          {state, units * head_dim * state_dim * 4}};
    const Span ins[] = {rows_range(x, batch, xl, x_stride, esz),
                         rows_range(B, batch, bl, b_stride, esz),
                         rows_range(C, batch, bl, c_stride, esz),
                         {dt, units * 4},
                         {A, (uint64_t)num_heads * 4},
                         {D, (uint64_t)num_heads * 4}};
    if ((st = check_alias(outs, ins)) != KDA_OK) return st;
    if (units == 0) return KDA_OK;
    if ((st = check_device()) != KDA_OK) return st;
    const kda::SsmStep a = {x, B, C, dt, A, D, state, out, batch, num_heads, num_groups,
                            head_dim, state_dim, x_stride, b_stride, c_stride, out_stride};
    return launch_status(kda::launch_ssm_step(a, dtype, stream), stream, "kda_ssm_decode_step");
}

}  // extern "C"
