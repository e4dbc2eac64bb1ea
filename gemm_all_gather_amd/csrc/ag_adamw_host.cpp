// Host side of the AdamW optimizer: the handle with its device table,
// validation and launches.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <memory>
#include <new>
#include <utility>
#include <vector>

#include "ag.h"
#include "ag_adamw.h"
#include "ag_status.h"

using ag::fail;
using ag::fail_hip;
using ag::ok;

struct ag_adamw {
    void* table = nullptr;              // device: the entries, then (256-byte aligned) the chunks
    uint64_t chunks_offset = 0;
    int64_t chunks = 0;
    std::vector<int64_t> sizes;
    int param = 0, grad = 0;
    bool master = false, state8 = false;
    int device = 0;

    ~ag_adamw()
    {
        if (table) (void)hipFree(table);
    }
};

namespace {

int bytes_of(int dtype)
{
    return dtype == AG_F32 ? 4 : dtype == AG_F16 || dtype == AG_BF16 ? 2 : 0;
}

ag_status_t check_pointer(const void* p, int64_t bytes, int align, const char* name, int64_t i, bool wanted)
{
    if (!wanted) return p == nullptr ? AG_OK : fail(AG_ERR_INVALID_ARG, "tensor %lld: %s is not NULL", static_cast<long long>(i), name);
    if (bytes == 0) return AG_OK;
    if (p == nullptr) return fail(AG_ERR_INVALID_ARG, "tensor %lld: %s is NULL", static_cast<long long>(i), name);
    if (reinterpret_cast<uint64_t>(p) % align != 0)
        return fail(AG_ERR_INVALID_ARG, "tensor %lld: %s is not aligned to %d bytes", static_cast<long long>(i), name, align);
    return AG_OK;
}

struct Range {
    uint64_t at, end;
    int64_t tensor;
    bool written;
    bool operator<(const Range& o) const { return at < o.at; }
};

ag_status_t create(const ag_adamw_tensor_t* tensors, int64_t count, ag_dtype_t param, ag_dtype_t grad, int bits, ag_adamw_t** out)
{
    if (!out) return fail(AG_ERR_INVALID_ARG, "out is NULL");
    if (!tensors) return fail(AG_ERR_INVALID_ARG, "tensors is NULL");
    if (count < 1 || count > (int64_t{1} << 20)) return fail(AG_ERR_INVALID_ARG, "count %lld not in [1, 2^20]", static_cast<long long>(count));
    if (bytes_of(param) == 0 || bytes_of(grad) == 0) return fail(AG_ERR_INVALID_ARG, "unknown param_dtype %d or grad_dtype %d", param, grad);
    if (bits != 32 && bits != 8) return fail(AG_ERR_INVALID_ARG, "state_bits %d is neither 32 nor 8", bits);
    auto h = std::make_unique<ag_adamw>();
    h->param = param;
    h->grad = grad;
    h->state8 = bits == 8;
    // the first tensor with elements says whether there are master weights
    for (int64_t i = 0; i < count; ++i)
        if (tensors[i].n > 0) {
            h->master = tensors[i].master != nullptr;
            break;
        }
    if (h->master && param == AG_F32) return fail(AG_ERR_UNSUPPORTED, "master weights with an fp32 param_dtype");
    const int sb = h->state8 ? 1 : 4;
    std::vector<ag::AdamwEntry> entries(static_cast<size_t>(count));
    std::vector<Range> ranges;
    int64_t blocks = 0, total = 0;
    for (int64_t i = 0; i < count; ++i) {
        const ag_adamw_tensor_t& t = tensors[i];
        if (t.n < 0) return fail(AG_ERR_INVALID_ARG, "tensor %lld: n %lld < 0", static_cast<long long>(i), static_cast<long long>(t.n));
        if (t.n >= (int64_t{1} << 40) || (total += t.n) >= (int64_t{1} << 40))
            return fail(AG_ERR_INVALID_ARG, "2^40 elements or more");
        const int64_t nb = (t.n + AG_ADAMW_BLOCK - 1) / AG_ADAMW_BLOCK;
        const struct { const void* p; int64_t bytes; int align; const char* name; bool wanted, written; } fields[] = {
            {t.param, t.n * bytes_of(param), bytes_of(param), "param", true, true},
            {t.grad, t.n * bytes_of(grad), bytes_of(grad), "grad", true, false},
            {t.exp_avg, t.n * sb, sb, "exp_avg", true, true},
            {t.exp_avg_sq, t.n * sb, sb, "exp_avg_sq", true, true},
            {t.exp_avg_scale, nb * 4, 4, "exp_avg_scale", h->state8, true},
            {t.exp_avg_sq_scale, nb * 4, 4, "exp_avg_sq_scale", h->state8, true},
            {t.master, t.n * 4, 4, "master", h->master, true},
        };
        for (const auto& f : fields) {
            if (t.n == 0) continue;
            const ag_status_t s = check_pointer(f.p, f.bytes, f.align, f.name, i, f.wanted);
            if (s != AG_OK) return s;
            if (f.wanted) {
                const uint64_t at = reinterpret_cast<uint64_t>(f.p);
                ranges.push_back(Range{at, at + static_cast<uint64_t>(f.bytes), i, f.written});
            }
        }
        entries[static_cast<size_t>(i)] = ag::AdamwEntry{t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale,
                                                         t.exp_avg_sq_scale, t.master, t.n, blocks};
        blocks += nb;
        h->chunks += (t.n + ag::kAdamwChunk - 1) / ag::kAdamwChunk;
        h->sizes.push_back(t.n);
    }
    // what is written may share no byte with anything else (gradients may be shared among themselves)
    std::sort(ranges.begin(), ranges.end());
    uint64_t written_end = 0, any_end = 0;
    int64_t written_by = -1, any_by = -1;
    for (const Range& r : ranges) {
        const uint64_t limit = r.written ? any_end : written_end;
        if (r.at < limit)
            return fail(AG_ERR_INVALID_ARG, "tensors %lld and %lld overlap", static_cast<long long>(r.written ? any_by : written_by),
                        static_cast<long long>(r.tensor));
        if (r.written && r.end > written_end) { written_end = r.end; written_by = r.tensor; }
        if (r.end > any_end) { any_end = r.end; any_by = r.tensor; }
    }
    if (h->chunks > 0x7fffffff) return fail(AG_ERR_UNSUPPORTED, "more than 2^31 chunks of %d elements", ag::kAdamwChunk);

    hipError_t e = hipGetDevice(&h->device);
    if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
    h->chunks_offset = (sizeof(ag::AdamwEntry) * static_cast<uint64_t>(count) + 255) / 256 * 256;
    std::vector<char> host(h->chunks_offset + sizeof(ag::AdamwChunk) * static_cast<uint64_t>(h->chunks));
    std::copy_n(reinterpret_cast<const char*>(entries.data()), sizeof(ag::AdamwEntry) * entries.size(), host.data());
    auto* chunk = reinterpret_cast<ag::AdamwChunk*>(host.data() + h->chunks_offset);
    for (int64_t i = 0; i < count; ++i)
        for (int64_t at = 0; at < tensors[i].n; at += ag::kAdamwChunk)
            *chunk++ = ag::AdamwChunk{static_cast<uint32_t>(i), static_cast<uint32_t>(at / ag::kAdamwChunk)};
    e = hipMalloc(&h->table, host.size());
    if (e != hipSuccess) {
        h->table = nullptr;
        return fail_hip(e, "hipMalloc(adamw table)");
    }
    e = hipMemcpy(h->table, host.data(), host.size(), hipMemcpyHostToDevice);
    if (e != hipSuccess) return fail_hip(e, "hipMemcpy(adamw table)");
    *out = h.release();
    return ok();
}

ag_status_t check_device(const ag_adamw_t* h)
{
    int dev = -1;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
    if (dev != h->device)
        return fail(AG_ERR_INVALID_ARG, "the optimizer's table lives on device %d but device %d is current", h->device, dev);
    return AG_OK;
}

ag_status_t check_hyper(const ag_adamw_hyper_t* y)
{
    if (!y) return fail(AG_ERR_INVALID_ARG, "hyper is NULL");
    for (int32_t r : y->reserved)
        if (r != 0) return fail(AG_ERR_INVALID_ARG, "a reserved field is not 0");
    if (!(y->beta1 >= 0 && y->beta1 < 1 && y->beta2 >= 0 && y->beta2 < 1)) return fail(AG_ERR_INVALID_ARG, "beta1 or beta2 not in [0, 1)");
    if (!(y->eps > 0) || !std::isfinite(y->eps) || static_cast<float>(y->eps) == 0.f) return fail(AG_ERR_INVALID_ARG, "eps is not positive in fp32");
    if (!std::isfinite(y->lr) || !std::isfinite(y->weight_decay) || !std::isfinite(y->grad_scale))
        return fail(AG_ERR_INVALID_ARG, "lr, weight_decay or grad_scale is not finite");
    if (y->step < 1) return fail(AG_ERR_INVALID_ARG, "step %lld < 1", static_cast<long long>(y->step));
    if (y->stochastic != 0 && y->stochastic != 1) return fail(AG_ERR_INVALID_ARG, "stochastic %d is not 0 or 1", y->stochastic);
    return AG_OK;
}

}  // namespace

extern "C" {

ag_status_t ag_adamw_create(const ag_adamw_tensor_t* tensors, int64_t count, ag_dtype_t param_dtype, ag_dtype_t grad_dtype,
                            int state_bits, ag_adamw_t** out)
{
    try {
        return create(tensors, count, param_dtype, grad_dtype, state_bits, out);
    } catch (const std::exception&) {
        return fail(AG_ERR_OUT_OF_MEMORY, "host allocation of the optimizer's table failed");
    }
}

ag_status_t ag_adamw_destroy(ag_adamw_t* optimizer)
{
    delete optimizer;
    return ok();
}

ag_status_t ag_adamw_step(const ag_adamw_t* optimizer, const ag_adamw_hyper_t* y, void* stream)
{
    if (!optimizer) return fail(AG_ERR_INVALID_ARG, "optimizer is NULL");
    ag_status_t s = check_hyper(y);
    if (s != AG_OK) return s;
    if ((s = check_device(optimizer)) != AG_OK) return s;
    if (optimizer->chunks == 0) return ok();
    ag::AdamwLaunch l{};
    ag::AdamwArgs& a = l.args;
    a.entries = static_cast<const ag::AdamwEntry*>(optimizer->table);
    a.chunks = reinterpret_cast<const ag::AdamwChunk*>(static_cast<const char*>(optimizer->table) + optimizer->chunks_offset);
    a.beta1 = y->beta1;
    a.beta2 = y->beta2;
    a.one_minus_beta1 = 1.0 - y->beta1;
    a.one_minus_beta2 = 1.0 - y->beta2;
    a.lr = y->lr;
    a.weight_decay = y->weight_decay;
    a.grad_scale = y->grad_scale;
    a.bias1 = 1.0 - std::pow(y->beta1, static_cast<double>(y->step));
    a.bias2 = 1.0 - std::pow(y->beta2, static_cast<double>(y->step));
    a.scalars = ag::AdamwScalars{static_cast<float>(a.beta1), static_cast<float>(a.one_minus_beta1), static_cast<float>(a.beta2),
                                 static_cast<float>(a.one_minus_beta2), static_cast<float>(1.0 - a.lr * a.weight_decay),
                                 static_cast<float>(a.lr / a.bias1), static_cast<float>(1.0 / a.bias2),
                                 static_cast<float>(y->eps), static_cast<float>(a.grad_scale), ag::adamw_mix_seed(y->seed)};
    a.seed = y->seed;
    a.dev_step = y->dev_step;
    a.dev_lr = y->dev_lr;
    a.dev_grad_scale = y->dev_grad_scale;
    a.stochastic = y->stochastic;
    l.chunks = optimizer->chunks;
    l.param = optimizer->param;
    l.grad = optimizer->grad;
    l.master = optimizer->master;
    l.state8 = optimizer->state8;
    const hipError_t e = ag::launch_adamw(l, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : fail_hip(e, "adamw step");
}

ag_status_t ag_adamw_read_states(const ag_adamw_t* optimizer, float* const* exp_avg, float* const* exp_avg_sq, void* stream)
{
    if (!optimizer) return fail(AG_ERR_INVALID_ARG, "optimizer is NULL");
    if (!optimizer->state8) return fail(AG_ERR_INVALID_ARG, "the states of this optimizer are fp32 already");
    if (!exp_avg || !exp_avg_sq) return fail(AG_ERR_INVALID_ARG, "exp_avg or exp_avg_sq is NULL");
    const int64_t count = static_cast<int64_t>(optimizer->sizes.size());
    for (int64_t i = 0; i < count; ++i) {
        if (optimizer->sizes[i] == 0) continue;
        ag_status_t s = check_pointer(exp_avg[i], 4, 4, "exp_avg output", i, true);
        if (s == AG_OK) s = check_pointer(exp_avg_sq[i], 4, 4, "exp_avg_sq output", i, true);
        if (s != AG_OK) return s;
    }
    const ag_status_t s = check_device(optimizer);
    if (s != AG_OK) return s;
    constexpr int64_t kPerGroup = 256 * 8;
    for (int64_t first = 0; first < count;) {
        ag::AdamwReadArgs a{};
        a.entries = static_cast<const ag::AdamwEntry*>(optimizer->table) + first;
        int64_t groups = 0;
        while (a.count < ag::kAdamwReadTensors && first + a.count < count) {
            const int64_t i = first + a.count, g = (optimizer->sizes[i] + kPerGroup - 1) / kPerGroup;
            if (groups + g > 0x7fffffff) break;
            a.exp_avg[a.count] = exp_avg[i];
            a.exp_avg_sq[a.count] = exp_avg_sq[i];
            a.first_group[a.count] = static_cast<uint32_t>(groups);
            groups += g;
            ++a.count;
        }
        a.first_group[a.count] = static_cast<uint32_t>(groups);
        if (groups > 0) {
            const hipError_t e = ag::launch_adamw_read(a, static_cast<hipStream_t>(stream));
            if (e != hipSuccess) return fail_hip(e, "adamw read states");
        }
        first += a.count;
    }
    return ok();
}

}  // extern "C"
