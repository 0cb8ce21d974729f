// C ABI of the training operators: argument checks, the AdamW handle, and the
// kernels' launches.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>
#include <unordered_set>
#include <vector>

#include "../../include/zero_ops.h"
#include "beta_pow.h"
#include "ops_internal.h"

namespace {

thread_local char g_last_error[512] = "";

zero_status fail(zero_status s, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return s;
}

zero_status hip_fail(hipError_t e, const char* what)
{
    return fail(ZERO_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// A caller's enum field as the integer it holds, which may be no enumerator.
template <typename E>
int32_t enum_value(const E& e)
{
    static_assert(sizeof(E) == sizeof(int32_t), "32-bit enum");
    int32_t v;
    std::memcpy(&v, &e, sizeof(v));
    return v;
}

bool known_type(int32_t t) { return t == ZERO_FP16 || t == ZERO_BF16 || t == ZERO_FP32; }
int type_bytes(int32_t t) { return t == ZERO_FP32 ? 4 : 2; }
bool finite_pos(double x) { return std::isfinite(x) && x > 0.0; }

bool scale_ok(double s)
{
    if (!finite_pos(s)) return false;
    const float inv = (float)(1.0 / s);
    return std::isfinite(inv) && inv > 0.0f;
}

// ------------------------------------------------------------------ arrays

// `rows` runs of `run` bytes, `step` bytes apart.
struct Array {
    const char* name;
    const void* p;
    size_t rows, run, step, align;
    bool written;
    uintptr_t begin() const { return (uintptr_t)p; }
    uintptr_t end() const { return begin() + (rows - 1) * step + run; }
};

Array flat(const char* name, const void* p, size_t bytes, size_t align, bool written)
{
    return Array{name, p, 1, bytes, bytes, align, written};
}

Array table(const char* name, const void* p, int64_t rows, int64_t width, int64_t stride, int esz, bool written)
{
    return Array{name, p, (size_t)rows, (size_t)width * esz, (size_t)stride * esz, (size_t)esz, written};
}

bool empty(const Array& a) { return a.p == nullptr || a.rows == 0 || a.run == 0; }

bool overlap(const Array& a, const Array& b)
{
    if (!(a.begin() < b.end() && b.begin() < a.end())) return false;
    if (a.rows > 1 && b.rows > 1 && a.step == b.step) {
        // columns of one buffer: the runs' places within the common step
        const size_t d = a.begin() > b.begin() ? (a.begin() - b.begin()) % a.step
                                               : (a.step - (b.begin() - a.begin()) % a.step) % a.step;
        return d < b.run || d + a.run > a.step;
    }
    return true;
}

zero_status past_end(const Array& a, hipDeviceptr_t base, size_t size, const char* who)
{
    if (a.end() <= (uintptr_t)base + size) return ZERO_OK;
    return fail(ZERO_ERR_INVALID_ARG, "%s: %s runs %zu bytes past the end of its allocation", who, a.name,
                (size_t)(a.end() - ((uintptr_t)base + size)));
}

// The runtime's view of an array: memory of this device, and its range inside its
// allocation.  With one GPU in the system an allocation that the runtime knows can be
// of no other, and one question is enough (two for each of six arrays are half of a
// small call's time).
zero_status on_device(const Array& a, int dev, const char* who)
{
    static const bool alone = [] {
        int n = 0;
        return hipGetDeviceCount(&n) == hipSuccess && n == 1;
    }();
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    if (alone) {
        if (hipMemGetAddressRange(&base, &size, (hipDeviceptr_t)a.p) == hipSuccess) return past_end(a, base, size, who);
        (void)hipGetLastError();
    }
    hipPointerAttribute_t t;
    if (hipPointerGetAttributes(&t, a.p) != hipSuccess) {
        (void)hipGetLastError();
        return ZERO_OK;
    }
    if (t.type == hipMemoryTypeUnregistered)
        return fail(ZERO_ERR_INVALID_ARG, "%s: %s is not device-accessible memory (pageable host memory?)", who, a.name);
    if (t.type == hipMemoryTypeDevice) {
        if (t.device != dev)
            return fail(ZERO_ERR_INVALID_ARG, "%s: %s is memory of device %d, the current one is %d", who, a.name, t.device, dev);
        if (hipMemGetAddressRange(&base, &size, (hipDeviceptr_t)a.p) == hipSuccess) return past_end(a, base, size, who);
        (void)hipGetLastError();
    }
    return ZERO_OK;
}

// Host checks of a call's arrays: alignment, and that a written one overlaps no
// other (`same`: the one pair that may be the same array).
zero_status check_arrays(const Array* a, int n, const char* who, int same_a = -1, int same_b = -1)
{
    for (int i = 0; i < n; ++i) {
        if (empty(a[i])) continue;
        if ((uintptr_t)a[i].p % a[i].align)
            return fail(ZERO_ERR_INVALID_ARG, "%s: %s is not aligned to %zu bytes", who, a[i].name, a[i].align);
        for (int j = 0; j < i; ++j) {
            if (empty(a[j]) || !(a[i].written || a[j].written)) continue;
            if (i == same_b && j == same_a && a[i].p == a[j].p && (a[i].step == a[j].step || a[i].rows == 1)) continue;
            if (overlap(a[i], a[j]))
                return fail(ZERO_ERR_INVALID_ARG, "%s: %s overlaps %s", who, a[i].name, a[j].name);
        }
    }
    return ZERO_OK;
}

// The current device, the stream's, and where the arrays are.
zero_status check_place(const Array* a, int n, void* stream, const char* who)
{
    int dev = -1;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, who);
    if (stream) {
        int sd = -1;
        if (hipStreamGetDevice(static_cast<hipStream_t>(stream), &sd) != hipSuccess)
            (void)hipGetLastError();
        else if (sd != dev)
            return fail(ZERO_ERR_INVALID_ARG, "%s: the stream belongs to device %d but device %d is current", who, sd, dev);
    }
    for (int i = 0; i < n; ++i) {
        if (empty(a[i])) continue;
        if (const zero_status s = on_device(a[i], dev, who)) return s;
    }
    return ZERO_OK;
}

constexpr int64_t kMaxGrid = 0x7fffffff;
constexpr int64_t kMaxElements = (int64_t)1 << 38;     // of a handle: 4 TB with fp32 masters and moments

// ------------------------------------------------------------------ layer norm

zero_status check_norm(int64_t rows, int64_t width, int32_t type, int32_t affine, const char* who)
{
    if (!known_type(type)) return fail(ZERO_ERR_INVALID_ARG, "%s: unknown type %d", who, (int)type);
    if (affine != type && affine != ZERO_FP32)
        return fail(ZERO_ERR_INVALID_ARG, "%s: affine must be the type of x or ZERO_FP32", who);
    if (rows < 0) return fail(ZERO_ERR_INVALID_ARG, "%s: rows must be >= 0", who);
    if (width < 1) return fail(ZERO_ERR_INVALID_ARG, "%s: width must be >= 1", who);
    if (width > (1 << 24)) return fail(ZERO_ERR_UNSUPPORTED, "%s: width above 2^24", who);
    if (rows > kMaxGrid) return fail(ZERO_ERR_UNSUPPORTED, "%s: rows above 2^31 - 1", who);
    return ZERO_OK;
}

// A row stride: what it must cover, and that the array's bytes can be counted.
zero_status check_stride(int64_t stride, int64_t rows, int64_t width, const char* name, const char* who)
{
    if (stride < width) return fail(ZERO_ERR_INVALID_ARG, "%s: %s's stride is less than the width", who, name);
    if (rows > 1 && stride > (INT64_MAX / 8 - width) / (rows - 1))
        return fail(ZERO_ERR_INVALID_ARG, "%s: %s's stride is out of range", who, name);
    return ZERO_OK;
}

int64_t norm_workspace(int64_t rows, int64_t width) { return zo::norm_partial_rows(rows, width) * 2 * width * 4; }

// ------------------------------------------------------------------ AdamW

zero_status check_hparams(const zero_adam_hparams* hp, const char* who)
{
    if (!hp) return fail(ZERO_ERR_INVALID_ARG, "%s: hp is NULL", who);
    if (!(std::isfinite(hp->lr) && hp->lr >= 0.0)) return fail(ZERO_ERR_INVALID_ARG, "%s: lr must be finite and >= 0", who);
    if (!(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0) ||
        !((float)hp->beta1 < 1.0f) || !((float)hp->beta2 < 1.0f))
        return fail(ZERO_ERR_INVALID_ARG, "%s: betas must lie in [0, 1), also in fp32", who);
    if (!finite_pos(hp->eps) || (float)hp->eps <= 0.0f)
        return fail(ZERO_ERR_INVALID_ARG, "%s: eps must be > 0 in fp32", who);
    if (!(std::isfinite(hp->weight_decay) && hp->weight_decay >= 0.0))
        return fail(ZERO_ERR_INVALID_ARG, "%s: weight_decay must be finite and >= 0", who);
    if (hp->bias_correction != 0 && hp->bias_correction != 1)
        return fail(ZERO_ERR_INVALID_ARG, "%s: bias_correction must be 0 or 1", who);
    const int32_t mode = enum_value(hp->wd_mode);
    if (mode != ZERO_WD_DECOUPLED && mode != ZERO_WD_L2) return fail(ZERO_ERR_INVALID_ARG, "%s: unknown wd_mode %d", who, (int)mode);
    if (hp->initial_step < 0) return fail(ZERO_ERR_INVALID_ARG, "%s: initial_step must be >= 0", who);
    return ZERO_OK;
}

zero_status check_scale(const zero_loss_scale_cfg* ls, const char* who)
{
    if (!ls) return fail(ZERO_ERR_INVALID_ARG, "%s: ls is NULL", who);
    if (!scale_ok(ls->init_scale) || !scale_ok(ls->min_scale))
        return fail(ZERO_ERR_INVALID_ARG, "%s: init_scale and min_scale must be finite and > 0 with a finite, non-zero fp32 reciprocal", who);
    if (ls->dynamic != 0 && ls->dynamic != 1) return fail(ZERO_ERR_INVALID_ARG, "%s: dynamic must be 0 or 1", who);
    if (ls->growth_interval < 1) return fail(ZERO_ERR_INVALID_ARG, "%s: growth_interval must be >= 1", who);
    return ZERO_OK;
}

// The arrays of one tensor, host checks only; appended to `all`.
zero_status tensor_arrays(const zero_adamw_tensor& t, int32_t index, int bits, std::vector<Array>& all, const char* who)
{
    const int32_t type = enum_value(t.type);
    if (!known_type(type)) return fail(ZERO_ERR_INVALID_ARG, "%s: tensor %d has unknown type %d", who, index, (int)type);
    if (t.numel < 0) return fail(ZERO_ERR_INVALID_ARG, "%s: tensor %d has numel < 0", who, index);
    if (t.numel > kMaxElements) return fail(ZERO_ERR_UNSUPPORTED, "%s: tensor %d has more than 2^38 elements", who, index);
    if (!(std::isfinite(t.weight_decay))) return fail(ZERO_ERR_INVALID_ARG, "%s: tensor %d: weight_decay must be finite", who, index);
    if (!(std::isfinite(t.lr_scale) && t.lr_scale >= 0.0)) return fail(ZERO_ERR_INVALID_ARG, "%s: tensor %d: lr_scale must be finite and >= 0", who, index);
    const size_t n = (size_t)t.numel, e = type_bytes(type), blocks = (n + zo::kStateBlock - 1) / zo::kStateBlock;
    const bool small = bits == 8;
    if ((type == ZERO_FP32) != (t.param == nullptr) && n > 0)
        return fail(ZERO_ERR_INVALID_ARG, "%s: tensor %d: param goes with the 2-byte formats, and only with them", who, index);
    if (small != (t.exp_avg_exp != nullptr) && n > 0)
        return fail(ZERO_ERR_INVALID_ARG, "%s: tensor %d: exponents go with 8-bit moments, and only with them", who, index);
    if ((t.exp_avg_exp != nullptr) != (t.exp_avg_sq_exp != nullptr))
        return fail(ZERO_ERR_INVALID_ARG, "%s: tensor %d has the exponents of one moment only", who, index);
    if (n == 0) return ZERO_OK;
    if (!t.grad || !t.master || !t.exp_avg || !t.exp_avg_sq)
        return fail(ZERO_ERR_INVALID_ARG, "%s: tensor %d: grad, master, exp_avg or exp_avg_sq is NULL", who, index);
    all.push_back(flat("grad", t.grad, n * e, e, false));
    all.push_back(flat("master", t.master, n * 4, 4, true));
    if (t.param) all.push_back(flat("param", t.param, n * e, e, true));
    all.push_back(flat("exp_avg", t.exp_avg, n * (small ? 1 : 4), small ? 1 : 4, true));
    all.push_back(flat("exp_avg_sq", t.exp_avg_sq, n * (small ? 1 : 4), small ? 1 : 4, true));
    if (small) {
        all.push_back(flat("exp_avg_exp", t.exp_avg_exp, blocks, 1, true));
        all.push_back(flat("exp_avg_sq_exp", t.exp_avg_sq_exp, blocks, 1, true));
    }
    return ZERO_OK;
}

}  // namespace

struct zero_adamw_s {
    int device = -1;
    int32_t n = 0;
    int bits = 32;
    bool checked = true;
    double max_norm = 0.0;
    uint64_t seed = 0;
    zero_adam_hparams hp{};
    zero_loss_scale_cfg ls{};
    int64_t nchunks = 0, chunk = 0;
    void* ws = nullptr;
    zo::TensorEntry* tensors = nullptr;
    zo::ChunkEntry* chunks = nullptr;
    zo::AdamwState* state = nullptr;
    double* partial = nullptr;
    zo::AdamwState* host_state = nullptr;      // pinned
    std::vector<int64_t> numel;
    std::vector<int32_t> type;
    std::vector<Array> written;                // by address; they overlap no other
};

namespace {

std::mutex g_live_mu;
std::unordered_set<zero_adamw_s*> g_live;

bool live(zero_adamw_t h)
{
    std::lock_guard<std::mutex> lk(g_live_mu);
    return h != nullptr && g_live.count(h) != 0;
}

zero_status check_handle(zero_adamw_t h, void* stream, const char* who)
{
    if (!live(h)) return fail(ZERO_ERR_STATE, "%s: not a live handle", who);
    int cur = -1;
    const hipError_t e = hipGetDevice(&cur);
    if (e != hipSuccess) return hip_fail(e, who);
    if (cur != h->device)
        return fail(ZERO_ERR_STATE, "%s: the handle belongs to device %d but device %d is current", who, h->device, cur);
    return check_place(nullptr, 0, stream, who);
}

void release(zero_adamw_s* h)
{
    if (h->ws) (void)hipFree(h->ws);
    if (h->host_state) (void)hipHostFree(h->host_state);
    delete h;
}

zo::AdamwState state_of(const zero_adamw_s* h, int64_t t, double scale, int64_t good)
{
    zo::AdamwState d{};
    d.scale = d.last_scale = scale;
    d.pw1 = beta_pow(h->hp.beta1, t);
    d.pw2 = beta_pow(h->hp.beta2, t);
    d.t = t;
    d.good = good;
    d.inv_scale = d.upd_inv_scale = (float)(1.0 / scale);
    d.bc1 = d.bc2 = d.clip = 1.0f;
    return d;
}

zero_status read_state(zero_adamw_t h, void* stream, const char* who)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = hipMemcpyAsync(h->host_state, h->state, sizeof(zo::AdamwState), hipMemcpyDeviceToHost, s);
    if (e == hipSuccess) e = hipStreamSynchronize(s);
    return e == hipSuccess ? ZERO_OK : hip_fail(e, who);
}

// No exception leaves the library: the host containers' are the only ones.
template <typename F>
zero_status guarded(const char* who, F f)
{
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return fail(ZERO_ERR_OOM, "%s: out of host memory", who);
    } catch (...) {
        return fail(ZERO_ERR_HIP, "%s: unexpected host error", who);
    }
}

}  // namespace

extern "C" {

const char* zero_ops_last_error(void) { return g_last_error; }
int zero_ops_abi_version(void) { return ZERO_OPS_ABI_VERSION; }

zero_status zero_layernorm_forward(const void* x, int64_t x_stride, const void* weight, const void* bias, int64_t rows,
                                   int64_t width, zero_lp_dtype type, zero_lp_dtype affine, double eps, void* y,
                                   int64_t y_stride, float* mean, float* rstd, void* stream)
{
    const char* who = "zero_layernorm_forward";
    const int32_t t = enum_value(type), at = enum_value(affine);
    if (const zero_status s = check_norm(rows, width, t, at, who)) return s;
    if (!(std::isfinite(eps) && eps >= 0.0)) return fail(ZERO_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
    if (const zero_status s = check_stride(x_stride, rows, width, "x", who)) return s;
    if (const zero_status s = check_stride(y_stride, rows, width, "y", who)) return s;
    if (rows == 0) return ZERO_OK;
    if (!x || !y) return fail(ZERO_ERR_INVALID_ARG, "%s: x or y is NULL", who);
    const int e = type_bytes(t), ae = type_bytes(at);
    const Array a[] = {table("x", x, rows, width, x_stride, e, false), table("y", y, rows, width, y_stride, e, true),
                       flat("weight", weight, (size_t)width * ae, ae, false), flat("bias", bias, (size_t)width * ae, ae, false),
                       flat("mean", mean, (size_t)rows * 4, 4, true), flat("rstd", rstd, (size_t)rows * 4, 4, true)};
    if (const zero_status s = check_arrays(a, 6, who, 0, 1)) return s;
    if (const zero_status s = check_place(a, 6, stream, who)) return s;
    const zo::NormForward f{x, weight, bias, y, mean, rstd, rows, width, x_stride, y_stride, (float)eps};
    const hipError_t err = zo::norm_forward(f, t, at, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? ZERO_OK : hip_fail(err, who);
}

zero_status zero_layernorm_workspace(int64_t rows, int64_t width, int64_t* bytes)
{
    const char* who = "zero_layernorm_workspace";
    if (!bytes) return fail(ZERO_ERR_INVALID_ARG, "%s: bytes is NULL", who);
    if (const zero_status s = check_norm(rows, width, ZERO_FP32, ZERO_FP32, who)) return s;
    *bytes = norm_workspace(rows, width);
    return ZERO_OK;
}

zero_status zero_layernorm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride, const void* weight,
                                    const float* mean, const float* rstd, int64_t rows, int64_t width, zero_lp_dtype type,
                                    zero_lp_dtype affine, void* dx, int64_t dx_stride, void* dweight, void* dbias,
                                    void* workspace, int64_t workspace_bytes, void* stream)
{
    const char* who = "zero_layernorm_backward";
    const int32_t t = enum_value(type), at = enum_value(affine);
    if (const zero_status s = check_norm(rows, width, t, at, who)) return s;
    if (const zero_status s = check_stride(dy_stride, rows, width, "dy", who)) return s;
    if (const zero_status s = check_stride(x_stride, rows, width, "x", who)) return s;
    if (const zero_status s = check_stride(dx_stride, rows, width, "dx", who)) return s;
    const bool sums = dweight != nullptr || dbias != nullptr;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx))
        return fail(ZERO_ERR_INVALID_ARG, "%s: dy, x, mean, rstd or dx is NULL", who);
    if (rows == 0 && !sums) return ZERO_OK;
    const int64_t need = norm_workspace(rows, width);
    if (sums && (!workspace || workspace_bytes < need))
        return fail(ZERO_ERR_INVALID_ARG, "%s: the workspace has %lld bytes, %lld are needed", who,
                    (long long)(workspace ? workspace_bytes : 0), (long long)need);
    const int e = type_bytes(t), ae = type_bytes(at);
    const Array a[] = {table("dy", dy, rows, width, dy_stride, e, false), table("x", x, rows, width, x_stride, e, false),
                       table("dx", dx, rows, width, dx_stride, e, true), flat("weight", weight, (size_t)width * ae, ae, false),
                       flat("mean", mean, (size_t)rows * 4, 4, false), flat("rstd", rstd, (size_t)rows * 4, 4, false),
                       flat("dweight", dweight, (size_t)width * ae, ae, true), flat("dbias", dbias, (size_t)width * ae, ae, true),
                       flat("workspace", sums ? workspace : nullptr, (size_t)need, 16, true)};
    if (const zero_status s = check_arrays(a, 9, who)) return s;
    if (const zero_status s = check_place(a, 9, stream, who)) return s;
    const zo::NormBackward b{dy, x, weight, mean, rstd, dx, dweight, dbias, sums ? static_cast<float*>(workspace) : nullptr,
                             rows, width, dy_stride, x_stride, dx_stride};
    const hipError_t err = zo::norm_backward(b, t, at, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? ZERO_OK : hip_fail(err, who);
}

static zero_status check_loss_sizes(int64_t tokens, int64_t vocab, int64_t width, int64_t max_tokens, const char* who)
{
    if (tokens < 0 || vocab < 1 || width < 1)
        return fail(ZERO_ERR_INVALID_ARG, "%s: tokens must be >= 0, vocab and width >= 1", who);
    if (max_tokens < 0 || max_tokens > 65535) return fail(ZERO_ERR_INVALID_ARG, "%s: max_tokens outside [0, 65535]", who);
    if (width > (1 << 20)) return fail(ZERO_ERR_UNSUPPORTED, "%s: width above 2^20", who);
    if (vocab > (1 << 21) - 64) return fail(ZERO_ERR_UNSUPPORTED, "%s: vocab above 2^21 - 64", who);
    if (tokens > kMaxGrid) return fail(ZERO_ERR_UNSUPPORTED, "%s: tokens above 2^31 - 1", who);
    return ZERO_OK;
}

constexpr int64_t kDefaultTokens = 8192;

zero_status zero_vocab_loss_workspace(int64_t tokens, int64_t vocab, int64_t width, int64_t max_tokens, int32_t gradient,
                                      int64_t* bytes)
{
    const char* who = "zero_vocab_loss_workspace";
    if (!bytes) return fail(ZERO_ERR_INVALID_ARG, "%s: bytes is NULL", who);
    if (gradient != 0 && gradient != 1) return fail(ZERO_ERR_INVALID_ARG, "%s: gradient must be 0 or 1", who);
    if (const zero_status s = check_loss_sizes(tokens, vocab, width, max_tokens, who)) return s;
    *bytes = zo::loss_plan(tokens, vocab, width, max_tokens ? max_tokens : kDefaultTokens, gradient != 0).bytes;
    return ZERO_OK;
}

zero_status zero_vocab_loss(const zero_vocab_loss_desc* d, const void* hidden, const void* weight, const int64_t* targets,
                            float* losses, float* lse, float* loss, void* dhidden, void* dweight, void* workspace,
                            int64_t workspace_bytes, void* stream)
{
    const char* who = "zero_vocab_loss";
    if (!d) return fail(ZERO_ERR_INVALID_ARG, "%s: desc is NULL", who);
    const int32_t t = enum_value(d->type);
    if (!known_type(t)) return fail(ZERO_ERR_INVALID_ARG, "%s: unknown type %d", who, (int)t);
    if (t == ZERO_FP32) return fail(ZERO_ERR_UNSUPPORTED, "%s: hidden states and weight are of a 2-byte type", who);
    if (const zero_status s = check_loss_sizes(d->tokens, d->vocab, d->width, d->max_tokens, who)) return s;
    // (an infinite factor would make NaN of the gradients that are 0)
    if (!std::isfinite((float)d->grad_scale)) return fail(ZERO_ERR_INVALID_ARG, "%s: grad_scale must be finite in fp32", who);
    const bool gradient = dweight != nullptr;
    if (d->tokens > 0 && gradient != (dhidden != nullptr))
        return fail(ZERO_ERR_INVALID_ARG, "%s: dhidden and dweight are given both or neither", who);
    if (const zero_status s = check_stride(d->hidden_stride, d->tokens, d->width, "hidden", who)) return s;
    if (const zero_status s = check_stride(d->weight_stride, d->vocab, d->width, "weight", who)) return s;
    if (gradient) {
        if (const zero_status s = check_stride(d->dhidden_stride, d->tokens, d->width, "dhidden", who)) return s;
        if (const zero_status s = check_stride(d->dweight_stride, d->vocab, d->width, "dweight", who)) return s;
    }
    if (!loss || !weight || (d->tokens > 0 && (!hidden || !targets || !losses)))
        return fail(ZERO_ERR_INVALID_ARG, "%s: hidden, weight, targets, losses or loss is NULL", who);
    const zo::LossPlan plan = zo::loss_plan(d->tokens, d->vocab, d->width, d->max_tokens ? d->max_tokens : kDefaultTokens, gradient);
    if (!workspace || workspace_bytes < plan.bytes)
        return fail(ZERO_ERR_INVALID_ARG, "%s: the workspace has %lld bytes, %lld are needed", who,
                    (long long)(workspace ? workspace_bytes : 0), (long long)plan.bytes);
    const size_t n = (size_t)d->tokens;
    const Array a[] = {table("hidden", hidden, d->tokens, d->width, d->hidden_stride, 2, false),
                       table("weight", weight, d->vocab, d->width, d->weight_stride, 2, false),
                       flat("targets", targets, n * 8, 8, false), flat("losses", losses, n * 4, 4, true),
                       flat("lse", lse, n * 4, 4, true), flat("loss", loss, 4, 4, true),
                       table("dhidden", dhidden, d->tokens, d->width, d->dhidden_stride, 2, true),
                       table("dweight", dweight, d->vocab, d->width, d->dweight_stride, 2, true),
                       flat("workspace", workspace, (size_t)plan.bytes, 256, true)};
    if (const zero_status s = check_arrays(a, 9, who)) return s;
    if (const zero_status s = check_place(a, 9, stream, who)) return s;
    const zo::Loss l{hidden, weight, targets, losses, lse, loss, dhidden, dweight, static_cast<char*>(workspace),
                     d->hidden_stride, d->weight_stride, d->dhidden_stride, d->dweight_stride, d->ignore_index, d->grad_scale};
    const hipError_t err = zo::vocab_loss(l, plan, t, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? ZERO_OK : hip_fail(err, who);
}

zero_status zero_adamw_init(const zero_adamw_tensor* tensors, int32_t n, const zero_adam_hparams* hp,
                            const zero_loss_scale_cfg* ls, const zero_adamw_cfg* cfg, zero_adamw_t* out)
{
    const char* who = "zero_adamw_init";
    if (!tensors || !cfg || !out) return fail(ZERO_ERR_INVALID_ARG, "%s: NULL argument", who);
    *out = nullptr;
    if (n < 1) return fail(ZERO_ERR_INVALID_ARG, "%s: n must be >= 1", who);
    if (n > (1 << 20)) return fail(ZERO_ERR_UNSUPPORTED, "%s: more than 2^20 tensors", who);
    if (const zero_status s = check_hparams(hp, who)) return s;
    if (const zero_status s = check_scale(ls, who)) return s;
    if (cfg->state_bits != 32 && cfg->state_bits != 8) return fail(ZERO_ERR_INVALID_ARG, "%s: state_bits must be 32 or 8", who);
    if (cfg->checked != 0 && cfg->checked != 1) return fail(ZERO_ERR_INVALID_ARG, "%s: checked must be 0 or 1", who);
    if (!(std::isfinite(cfg->max_grad_norm) && cfg->max_grad_norm >= 0.0))
        return fail(ZERO_ERR_INVALID_ARG, "%s: max_grad_norm must be finite and >= 0", who);
    if (cfg->max_grad_norm > 0.0 && !cfg->checked) return fail(ZERO_ERR_INVALID_ARG, "%s: clipping needs checked = 1", who);
    return guarded(who, [&]() -> zero_status {
        std::vector<Array> all;
        std::vector<zo::TensorEntry> table((size_t)n);
        std::vector<zo::ChunkEntry> chunks;
        int64_t elements = 0;
        for (int32_t i = 0; i < n; ++i) {
            const zero_adamw_tensor& t = tensors[i];
            if (const zero_status s = tensor_arrays(t, i, cfg->state_bits, all, who)) return s;
            table[i] = zo::TensorEntry{t.grad, t.master, t.param, t.exp_avg, t.exp_avg_sq, t.exp_avg_exp, t.exp_avg_sq_exp,
                                       t.numel, (float)t.weight_decay, (float)t.lr_scale, enum_value(t.type), 0};
            elements += t.numel;
            if (elements > kMaxElements) return fail(ZERO_ERR_UNSUPPORTED, "%s: more than 2^38 elements", who);
        }
        // overlaps of so many arrays by their order in memory
        std::vector<const Array*> order;
        for (const Array& a : all) {
            if ((uintptr_t)a.p % a.align) return fail(ZERO_ERR_INVALID_ARG, "%s: a tensor's %s is not aligned to %zu bytes", who, a.name, a.align);
            order.push_back(&a);
        }
        std::sort(order.begin(), order.end(), [](const Array* a, const Array* b) { return a->begin() < b->begin(); });
        const Array* written = nullptr;      // the one that reaches furthest, of those written, and of all
        const Array* any = nullptr;
        for (const Array* a : order) {
            const Array* before = a->written ? any : written;
            if (before && before->end() > a->begin())
                return fail(ZERO_ERR_INVALID_ARG, "%s: a tensor's %s overlaps a tensor's %s", who, a->name, before->name);
            if (!any || a->end() > any->end()) any = a;
            if (a->written && (!written || a->end() > written->end())) written = a;
        }
        if (const zero_status s = check_place(all.data(), (int)all.size(), nullptr, who)) return s;
        const int64_t chunk = zo::adamw_chunk(elements);
        for (int32_t i = 0; i < n; ++i)
            for (int64_t b = 0; b < tensors[i].numel; b += chunk) chunks.push_back(zo::ChunkEntry{i, 0, b});
        zero_adamw_s* h = new zero_adamw_s;
        h->n = n;
        h->bits = cfg->state_bits;
        h->checked = cfg->checked != 0;
        h->max_norm = cfg->max_grad_norm;
        h->seed = cfg->seed;
        h->hp = *hp;
        h->ls = *ls;
        h->nchunks = (int64_t)chunks.size();
        h->chunk = chunk;
        const size_t bt = table.size() * sizeof(table[0]), bc = chunks.size() * sizeof(zo::ChunkEntry);
        auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
        hipError_t e = hipGetDevice(&h->device);
        if (e == hipSuccess) e = hipMalloc(&h->ws, up(bt) + up(bc) + up(2 * sizeof(zo::AdamwState)) + up(zo::kAdamwPartials * 8));
        if (e == hipSuccess) e = hipHostMalloc((void**)&h->host_state, sizeof(zo::AdamwState));
        if (e != hipSuccess) {
            release(h);
            (void)hipGetLastError();
            return fail(ZERO_ERR_OOM, "%s: workspace: %s", who, hipGetErrorString(e));
        }
        char* at = static_cast<char*>(h->ws);
        h->tensors = reinterpret_cast<zo::TensorEntry*>(at);
        h->chunks = reinterpret_cast<zo::ChunkEntry*>(at + up(bt));
        h->state = reinterpret_cast<zo::AdamwState*>(at + up(bt) + up(bc));
        h->partial = reinterpret_cast<double*>(at + up(bt) + up(bc) + up(2 * sizeof(zo::AdamwState)));
        const zo::AdamwState first = state_of(h, hp->initial_step, ls->init_scale, 0);
        e = hipMemcpy(h->tensors, table.data(), bt, hipMemcpyHostToDevice);
        if (e == hipSuccess && bc) e = hipMemcpy(h->chunks, chunks.data(), bc, hipMemcpyHostToDevice);
        if (e == hipSuccess) e = hipMemcpy(h->state, &first, sizeof(first), hipMemcpyHostToDevice);
        if (e != hipSuccess) {
            release(h);
            return hip_fail(e, who);
        }
        try {
            for (const zo::TensorEntry& t : table) {
                h->numel.push_back(t.numel);
                h->type.push_back(t.type);
            }
            for (const Array* a : order)
                if (a->written) h->written.push_back(*a);
            std::lock_guard<std::mutex> lk(g_live_mu);
            g_live.insert(h);
        } catch (...) {
            release(h);
            throw;
        }
        *out = h;
        return ZERO_OK;
    });
}

zero_status zero_adamw_set_grads(zero_adamw_t h, const void* const* grads, int32_t n, void* stream)
{
    const char* who = "zero_adamw_set_grads";
    if (const zero_status s = check_handle(h, stream, who)) return s;
    if (!grads || n != h->n) return fail(ZERO_ERR_INVALID_ARG, "%s: one gradient for each of the %d tensors is needed", who, (int)h->n);
    for (int32_t i = 0; i < n; ++i) {
        if (h->numel[i] == 0) continue;
        if (!grads[i]) return fail(ZERO_ERR_INVALID_ARG, "%s: gradient %d is NULL", who, (int)i);
        const int e = type_bytes(h->type[i]);
        const Array a = flat("a gradient", grads[i], (size_t)h->numel[i] * e, e, false);
        if (const zero_status s = check_arrays(&a, 1, who)) return s;
        const auto w = std::upper_bound(h->written.begin(), h->written.end(), a.begin(),
                                        [](uintptr_t at, const Array& x) { return at < x.end(); });
        if (w != h->written.end() && overlap(a, *w))
            return fail(ZERO_ERR_INVALID_ARG, "%s: gradient %d overlaps a tensor's %s", who, (int)i, w->name);
        if (const zero_status s = on_device(a, h->device, who)) return s;
    }
    for (int32_t i = 0; i < n; i += zo::kGradsPerLaunch) {
        const int count = n - i < zo::kGradsPerLaunch ? n - i : zo::kGradsPerLaunch;
        const hipError_t e = zo::adamw_set_grads(h->tensors, grads, i, count, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return hip_fail(e, who);
    }
    return ZERO_OK;
}

zero_status zero_adamw_step(zero_adamw_t h, const zero_adam_hparams* hp, void* stream)
{
    const char* who = "zero_adamw_step";
    if (const zero_status s = check_handle(h, stream, who)) return s;
    if (hp) {
        if (const zero_status s = check_hparams(hp, who)) return s;
        if (hp->beta1 != h->hp.beta1 || hp->beta2 != h->hp.beta2)
            return fail(ZERO_ERR_INVALID_ARG, "%s: the betas must be those of the handle", who);
    }
    const zero_adam_hparams& p = hp ? *hp : h->hp;
    zo::AdamwLaunch a{};
    a.tensors = h->tensors;
    a.chunks = h->chunks;
    a.nchunks = h->nchunks;
    a.chunk = h->chunk;
    a.state = h->state;
    a.partial = h->partial;
    a.s.b1 = (float)p.beta1;
    a.s.b2 = (float)p.beta2;
    a.s.omb1 = (float)(1.0 - (double)a.s.b1);
    a.s.omb2 = (float)(1.0 - (double)a.s.b2);
    a.s.eps = (float)p.eps;
    a.s.lr = (float)p.lr;
    a.s.wd = (float)p.weight_decay;
    a.s.b1d = (double)a.s.b1;
    a.s.b2d = (double)a.s.b2;
    a.s.min_scale = h->ls.min_scale;
    a.s.max_norm = h->max_norm;
    a.s.bias_correction = p.bias_correction;
    a.s.dynamic = h->ls.dynamic;
    a.s.growth_interval = h->ls.growth_interval;
    a.s.l2 = enum_value(p.wd_mode) == ZERO_WD_L2;
    a.s.seed = h->seed;
    const hipError_t e = zo::adamw_step(a, h->bits, h->checked, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ZERO_OK : hip_fail(e, who);
}

zero_status zero_adamw_result(zero_adamw_t h, void* stream, zero_step_info* out)
{
    const char* who = "zero_adamw_result";
    if (const zero_status s = check_handle(h, stream, who)) return s;
    if (!out) return fail(ZERO_ERR_INVALID_ARG, "%s: out is NULL", who);
    if (const zero_status s = read_state(h, stream, who)) return s;
    const zo::AdamwState& d = *h->host_state;
    out->overflow = d.skip;
    out->skipped = d.skip;
    out->step_t = d.t;
    out->grad_norm = std::sqrt(d.sumsq);
    out->scale_used = d.last_scale;
    out->scale_next = d.scale;
    return ZERO_OK;
}

zero_status zero_adamw_get_counters(zero_adamw_t h, void* stream, int64_t* step_t, double* scale, int64_t* good_steps)
{
    const char* who = "zero_adamw_get_counters";
    if (const zero_status s = check_handle(h, stream, who)) return s;
    if (!step_t || !scale || !good_steps) return fail(ZERO_ERR_INVALID_ARG, "%s: NULL argument", who);
    if (const zero_status s = read_state(h, stream, who)) return s;
    *step_t = h->host_state->t;
    *scale = h->host_state->scale;
    *good_steps = h->host_state->good;
    return ZERO_OK;
}

zero_status zero_adamw_set_counters(zero_adamw_t h, void* stream, int64_t step_t, double scale, int64_t good_steps)
{
    const char* who = "zero_adamw_set_counters";
    if (const zero_status s = check_handle(h, stream, who)) return s;
    if (step_t < 0 || good_steps < 0 || !scale_ok(scale))
        return fail(ZERO_ERR_INVALID_ARG, "%s: step_t and good_steps must be >= 0, scale as init_scale", who);
    const hipError_t e = zo::adamw_set_state(h->state, state_of(h, step_t, scale, good_steps), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ZERO_OK : hip_fail(e, who);
}

zero_status zero_adamw_destroy(zero_adamw_t h)
{
    {
        std::lock_guard<std::mutex> lk(g_live_mu);
        if (!h || !g_live.erase(h)) return fail(ZERO_ERR_STATE, "zero_adamw_destroy: not a live handle");
    }
    release(h);      // hipFree waits for the device
    return ZERO_OK;
}

zero_status zero_moments_pack(const float* x, int64_t n, int32_t is_signed, uint8_t* codes, int8_t* exps, void* stream)
{
    const char* who = "zero_moments_pack";
    if (n < 0 || n > ((int64_t)1 << 40)) return fail(ZERO_ERR_INVALID_ARG, "%s: n outside [0, 2^40]", who);
    if (is_signed != 0 && is_signed != 1) return fail(ZERO_ERR_INVALID_ARG, "%s: is_signed must be 0 or 1", who);
    if (n == 0) return ZERO_OK;
    if (!x || !codes || !exps) return fail(ZERO_ERR_INVALID_ARG, "%s: NULL array", who);
    const size_t blocks = ((size_t)n + zo::kStateBlock - 1) / zo::kStateBlock;
    const Array a[] = {flat("x", x, (size_t)n * 4, 4, false), flat("codes", codes, (size_t)n, 1, true), flat("exps", exps, blocks, 1, true)};
    if (const zero_status s = check_arrays(a, 3, who)) return s;
    if (const zero_status s = check_place(a, 3, stream, who)) return s;
    const hipError_t e = zo::moments_pack(x, codes, exps, n, is_signed != 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ZERO_OK : hip_fail(e, who);
}

zero_status zero_moments_unpack(const uint8_t* codes, const int8_t* exps, int64_t n, int32_t is_signed, zero_lp_dtype out_type,
                                void* out, void* stream)
{
    const char* who = "zero_moments_unpack";
    const int32_t t = enum_value(out_type);
    if (n < 0 || n > ((int64_t)1 << 40)) return fail(ZERO_ERR_INVALID_ARG, "%s: n outside [0, 2^40]", who);
    if (is_signed != 0 && is_signed != 1) return fail(ZERO_ERR_INVALID_ARG, "%s: is_signed must be 0 or 1", who);
    if (t != ZERO_FP32 && t != ZERO_BF16) return fail(ZERO_ERR_INVALID_ARG, "%s: out_type must be ZERO_FP32 or ZERO_BF16", who);
    if (n == 0) return ZERO_OK;
    if (!out || !codes || !exps) return fail(ZERO_ERR_INVALID_ARG, "%s: NULL array", who);
    const size_t blocks = ((size_t)n + zo::kStateBlock - 1) / zo::kStateBlock;
    const int e = type_bytes(t);
    const Array a[] = {flat("codes", codes, (size_t)n, 1, false), flat("exps", exps, blocks, 1, false), flat("out", out, (size_t)n * e, e, true)};
    if (const zero_status s = check_arrays(a, 3, who)) return s;
    if (const zero_status s = check_place(a, 3, stream, who)) return s;
    const hipError_t err = zo::moments_unpack(codes, exps, out, n, t, is_signed != 0, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? ZERO_OK : hip_fail(err, who);
}

}  // extern "C"
