// kv_api.cpp -- C entry points of the quantised cache, the shared-prefix
// attention over it, the draft verification and the log probabilities
// (include/lora.h): argument checks, handles and their memory, launches.  As with the pools, nothing on
// the hot path allocates or waits.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <exception>
#include <new>

#include "../../include/lora.h"
#include "attend_plan.hpp"
#include "host.hpp"
#include "kv_internal.hpp"

using lora::align_up;
using lora::alloc_status;
using lora::aligned;
using lora::DeviceGuard;
using lora::hip_fail;

static_assert(LORA_VERIFY_MAX_VOCAB == lora::VERIFY_PART * lora::VERIFY_PARTS, "a lane for each part of a row");
static_assert(LORA_SCORE_MAX_TOP == lora::LOGPROBS_MAX_TOP, "the kernels have room for so many");
static_assert(LORA_VERIFY_MAX_VOCAB == 256 * 128 * lora::LOGPROBS_MAX_PARTS, "a part is 32768 logits, or the whole row");
static_assert(LORA_ROPE_MAX_AXES == lora::ROPE_MAX_AXES, "the kernels keep the positions of so many");
static_assert(LORA_VERIFY_MAX_VOCAB == lora::VERIFY_CHUNKS * lora::VERIFY_MAX_SEGMENTS * 512, "a lane for each segment");
static_assert(LORA_VERIFY_MAX_DRAFTS == lora::VERIFY_MAX_DRAFTS, "a lane for each drafted token");

struct lora_kv_s {
    int device = 0;
    int page_size = 0;
    lora::KvCache c{};
    char *mem = nullptr;
};

struct lora_rope_s {
    int device = 0;
    char *mem = nullptr;
    lora::RopeTable t{};
};

struct lora_attend_plan_s {
    int device = 0;
    int max_tokens = 0, n_heads = 0, n_kv_heads = 0, head_dim = 0;
    lora::AttendPlanner planner;
    char *mem = nullptr;                    // the plan as the kernels read it, then the partial results
    float *part_o = nullptr, *part_ml = nullptr;
    unsigned *count = nullptr;
    // Two pinned copies of the plan: one may still be on its way to the device
    // while the next is written.
    void *host[2] = {nullptr, nullptr};
    hipEvent_t sent[2] = {nullptr, nullptr};
    int next = 0;
    bool set = false;
    int sent_tokens = -1;  // of the last plan that went to the device; -1: none did
    int page_size = 0, n_pages = 0;
    std::mutex mu;

    lora_attend_plan_s(int seqs, int groups, int tokens, int pages, int heads, int kv_heads)
        : planner(seqs, groups, tokens, pages, heads, kv_heads) {}
};

struct lora_scorer_s {
    int device = 0;
    int max_rows = 0;
    char *mem = nullptr;
    uint64_t *keys = nullptr;
    float *stats = nullptr;
    unsigned *count = nullptr;
};

struct lora_verifier_s {
    int device = 0;
    int max_seqs = 0;
    char *mem = nullptr;
    double *sums = nullptr;
    unsigned *count = nullptr;
    double *row_sums = nullptr;
    unsigned *row_count = nullptr;
};

namespace {

bool dim_ok(int d) { return d == 64 || d == 128; }

// Waits for the device's work and frees `mem` on its device.
int free_on(int device, char *mem) {
    DeviceGuard g(device);
    HIP_TRY(g.error());
    const hipError_t e = hipDeviceSynchronize();
    (void)hipFree(mem);
    return e == hipSuccess ? LORA_OK : hip_fail(e);
}

void free_plan(lora_attend_plan p) {
    for (int i = 0; i < 2; ++i) {
        if (p->host[i]) (void)hipHostFree(p->host[i]);
        if (p->sent[i]) (void)hipEventDestroy(p->sent[i]);
    }
    if (p->mem) (void)hipFree(p->mem);
}

// What lora_kv_write and lora_kv_append ask of their keys and values.
bool rows_ok(const lora_kv_s *kv, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
             const int32_t *slots) {
    const int64_t row = static_cast<int64_t>(kv->c.heads) * kv->c.dim;
    return k != nullptr && v != nullptr && slots != nullptr && k_stride >= row && v_stride >= row && aligned(k, 16) &&
           aligned(v, 16) && aligned(slots, 4) && k_stride % 8 == 0 && v_stride % 8 == 0;
}

// Checks and cuts a batch on the host.  tree: `parent` has to be there, if there
// are new tokens.
int plan_batch(lora_attend_plan plan, lora_kv kv, const lora_attend_batch *batch, const int32_t *parent, bool tree) {
    if (kv == nullptr || batch == nullptr) return LORA_EINVAL;
    if (kv->device != plan->device || kv->c.heads != plan->n_kv_heads || kv->c.dim != plan->head_dim)
        return LORA_EMISMATCH;
    const lora::AttendBatch b{batch->n_seqs, batch->n_groups, batch->q_len, batch->kv_len, batch->group,
                              batch->pages, batch->page0, batch->prefix_len, batch->prefix_pages,
                              batch->prefix_page0, parent, tree};
    return plan->planner.plan(b, lora::AttendGeometry{plan->n_heads, plan->n_kv_heads, kv->page_size, kv->c.n_pages});
}

// The plan of a batch, to the device.
int set_plan(lora_attend_plan plan, lora_kv kv, const lora_attend_batch *batch, const int32_t *parent, bool tree,
             void *stream) {
    if (plan == nullptr) return LORA_EINVAL;
    std::lock_guard<std::mutex> lk(plan->mu);
    plan->set = false;  // until this batch is on its way, whatever refuses it
    DeviceGuard g(plan->device);
    HIP_TRY(g.error());
    hipStream_t st = static_cast<hipStream_t>(stream);
    // A captured copy would send whatever the pinned buffer holds at replay.
    hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
    HIP_TRY(hipStreamIsCapturing(st, &cap));
    if (cap != hipStreamCaptureStatusNone) return LORA_EINVAL;
    const int rc = plan_batch(plan, kv, batch, parent, tree);
    // A refused batch leaves the device a plan for no cache, so that graphs do
    // not attend to the one before.
    if (rc != LORA_OK && plan->sent_tokens < 0) return rc;
    const int i = plan->next;
    HIP_TRY(hipEventSynchronize(plan->sent[i]));  // done at once unless two plans are still on their way
    const size_t bytes = rc == LORA_OK ? plan->planner.write(plan->host[i])
                                       : lora::AttendPlanner::write_none(plan->host[i], plan->sent_tokens);
    HIP_TRY(hipMemcpyAsync(plan->mem, plan->host[i], bytes, hipMemcpyHostToDevice, st));
    HIP_TRY(hipEventRecord(plan->sent[i], st));
    plan->next = 1 - i;
    if (rc != LORA_OK) return rc;
    plan->sent_tokens = static_cast<int>(plan->planner.tokens().size());
    plan->page_size = kv->page_size;
    plan->n_pages = kv->c.n_pages;
    plan->set = true;
    return LORA_OK;
}

}  // namespace

extern "C" {

int lora_kv_create(int n_pages, int page_size, int n_kv_heads, int head_dim, lora_dtype dtype, lora_kv *out) {
    if (out == nullptr) return LORA_EINVAL;
    *out = nullptr;
    if (n_pages < 1 || n_kv_heads < 1 || n_kv_heads > LORA_KV_MAX_HEADS || !dim_ok(head_dim)) return LORA_EINVAL;
    if (page_size < 16 || page_size > LORA_KV_MAX_PAGE || (page_size & (page_size - 1)) != 0) return LORA_EINVAL;
    if (dtype != LORA_F16 && dtype != LORA_BF16) return LORA_EINVAL;
    // A slot is an int32.
    if (static_cast<int64_t>(n_pages) * page_size > 0x7FFFFFFF) return LORA_EINVAL;
    lora_kv kv = new (std::nothrow) lora_kv_s;
    if (kv == nullptr) return LORA_ENOMEM;
    int shift = 0;
    while ((1 << shift) < page_size) ++shift;
    const size_t rows = static_cast<size_t>(n_pages) * page_size * n_kv_heads;
    const size_t elems = align_up(rows * head_dim, 256), exps = align_up(rows, 256);
    const size_t total = 2 * elems + 2 * exps + 256;
    hipError_t e = hipGetDevice(&kv->device);
    if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void **>(&kv->mem), total);
    if (e != hipSuccess) {
        const int rc = alloc_status(e);
        delete kv;
        return rc;
    }
    kv->page_size = page_size;
    kv->c = lora::KvCache{reinterpret_cast<uint8_t *>(kv->mem),
                          reinterpret_cast<uint8_t *>(kv->mem + elems),
                          reinterpret_cast<uint8_t *>(kv->mem + 2 * elems),
                          reinterpret_cast<uint8_t *>(kv->mem + 2 * elems + exps),
                          reinterpret_cast<unsigned long long *>(kv->mem + 2 * elems + 2 * exps),
                          n_pages, shift, n_kv_heads, head_dim, static_cast<int>(dtype)};
    // A row that was never written is a row of zeros.
    e = hipMemset(kv->mem, 0, total);
    if (e == hipSuccess) e = hipMemset(kv->c.kexp, lora::KV_EXP_BIAS + lora::KV_MIN_EXP, exps);
    if (e == hipSuccess) e = hipMemset(kv->c.vinv, lora::KV_EXP_BIAS - lora::KV_MIN_EXP, exps);
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) {
        const int rc = hip_fail(e);
        (void)hipFree(kv->mem);
        delete kv;
        return rc;
    }
    *out = kv;
    return LORA_OK;
}

int lora_kv_destroy(lora_kv kv) {
    if (kv == nullptr) return LORA_OK;
    const int rc = free_on(kv->device, kv->mem);
    delete kv;
    return rc;
}

int lora_kv_write(lora_kv kv, const void *k, int64_t k_stride, const void *v, int64_t v_stride, const int32_t *slots,
                  int n_tokens, void *stream) {
    if (kv == nullptr || n_tokens < 0) return LORA_EINVAL;
    if (n_tokens == 0) return LORA_OK;
    if (!rows_ok(kv, k, k_stride, v, v_stride, slots)) return LORA_EINVAL;
    DeviceGuard g(kv->device);
    HIP_TRY(g.error());
    HIP_TRY(lora::launch_kv_write(kv->c, k, k_stride, v, v_stride, slots, n_tokens, static_cast<hipStream_t>(stream)));
    return LORA_OK;
}

int lora_kv_read(lora_kv kv, const int32_t *slots, int n_tokens, void *k, void *v, void *stream) {
    if (kv == nullptr || n_tokens < 0) return LORA_EINVAL;
    if (n_tokens == 0) return LORA_OK;
    if (k == nullptr || v == nullptr || slots == nullptr || k == v) return LORA_EINVAL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return LORA_EINVAL;
    DeviceGuard g(kv->device);
    HIP_TRY(g.error());
    HIP_TRY(lora::launch_kv_read(kv->c, slots, n_tokens, k, v, static_cast<hipStream_t>(stream)));
    return LORA_OK;
}

int lora_rope_create(int n_positions, int rot_dim, const double *freq, const int32_t *axis, int n_axes, int pairs,
                     double scale, lora_rope *out) {
    if (out == nullptr) return LORA_EINVAL;
    *out = nullptr;
    if (n_positions < 1 || n_positions > LORA_ROPE_MAX_POSITIONS || n_axes < 1 || n_axes > LORA_ROPE_MAX_AXES)
        return LORA_EINVAL;
    if (rot_dim < 16 || rot_dim > 128 || rot_dim % 16 != 0 || freq == nullptr) return LORA_EINVAL;
    if (!(scale > 0.0 && scale <= 1024.0)) return LORA_EINVAL;
    const int n = rot_dim / 2;
    int32_t axes[64] = {};
    for (int i = 0; i < n; ++i) {
        // Nor may the farthest angle overflow: it has no cosine.
        if (!std::isfinite(freq[i]) || !std::isfinite(freq[i] * (n_positions - 1))) return LORA_EINVAL;
        if (axis != nullptr) axes[i] = axis[i];
        if (axes[i] < 0 || axes[i] >= n_axes) return LORA_EINVAL;
    }
    lora_rope r = new (std::nothrow) lora_rope_s;
    if (r == nullptr) return LORA_ENOMEM;
    const size_t half = align_up(static_cast<size_t>(n_positions) * n * sizeof(float2), 256);
    const size_t total = 2 * half + 64 * sizeof(int32_t) + 64 * sizeof(double);
    hipError_t e = hipGetDevice(&r->device);
    if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void **>(&r->mem), total);
    if (e != hipSuccess) {
        const int rc = alloc_status(e);
        delete r;
        return rc;
    }
    float2 *hi = reinterpret_cast<float2 *>(r->mem), *lo = reinterpret_cast<float2 *>(r->mem + half);
    int32_t *axis_dev = reinterpret_cast<int32_t *>(r->mem + 2 * half);
    double *freq_dev = reinterpret_cast<double *>(r->mem + 2 * half + 64 * sizeof(int32_t));
    e = hipMemcpy(axis_dev, axes, static_cast<size_t>(n) * sizeof(int32_t), hipMemcpyHostToDevice);
    if (e == hipSuccess) e = hipMemcpy(freq_dev, freq, static_cast<size_t>(n) * sizeof(double), hipMemcpyHostToDevice);
    if (e == hipSuccess) e = lora::launch_rope_table(freq_dev, scale, n_positions, n, hi, lo, nullptr);
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) {
        const int rc = hip_fail(e);
        (void)hipFree(r->mem);
        delete r;
        return rc;
    }
    r->t = lora::RopeTable{hi, lo, axis_dev, n_positions, n, n_axes, pairs != 0};
    *out = r;
    return LORA_OK;
}

int lora_rope_destroy(lora_rope rope) {
    if (rope == nullptr) return LORA_OK;
    const int rc = free_on(rope->device, rope->mem);
    delete rope;
    return rc;
}

int lora_kv_append(lora_kv kv, lora_rope rope, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                   const int32_t *slots, const int32_t *positions, int n_tokens, const void *q, int64_t q_stride,
                   int n_heads, void *q_out, int64_t q_out_stride, void *stream) {
    if (kv == nullptr || rope == nullptr || n_tokens < 0) return LORA_EINVAL;
    if (rope->device != kv->device || 2 * rope->t.n > kv->c.dim) return LORA_EMISMATCH;
    if (n_tokens == 0) return LORA_OK;
    if (!rows_ok(kv, k, k_stride, v, v_stride, slots)) return LORA_EINVAL;
    if (positions == nullptr || !aligned(positions, 4)) return LORA_EINVAL;
    lora::TurnArgs a{};
    a.t = rope->t;
    a.positions = positions;
    if (q != nullptr) {
        if (n_heads < 1 || n_heads > LORA_KV_MAX_HEADS * lora::ATTEND_MAX_GQ) return LORA_EINVAL;
        const int64_t row = static_cast<int64_t>(n_heads) * kv->c.dim;
        if (q_out == nullptr || !aligned(q, 16) || !aligned(q_out, 16)) return LORA_EINVAL;
        if (q_stride < row || q_out_stride < row || q_stride % 8 != 0 || q_out_stride % 8 != 0) return LORA_EINVAL;
        if (q == q_out && q_stride != q_out_stride) return LORA_EINVAL;
        a.q = static_cast<const uint16_t *>(q);
        a.q_out = static_cast<uint16_t *>(q_out);
        a.q_stride = q_stride;
        a.out_stride = q_out_stride;
        a.n_heads = n_heads;
    }
    DeviceGuard g(kv->device);
    HIP_TRY(g.error());
    HIP_TRY(lora::launch_kv_append(kv->c, a, k, k_stride, v, v_stride, slots, n_tokens, static_cast<hipStream_t>(stream)));
    return LORA_OK;
}

int lora_kv_poll_errors(lora_kv kv, uint64_t *n_invalid_slots) {
    if (kv == nullptr || n_invalid_slots == nullptr) return LORA_EINVAL;
    DeviceGuard g(kv->device);
    HIP_TRY(g.error());
    HIP_TRY(hipDeviceSynchronize());
    unsigned long long n = 0;
    HIP_TRY(hipMemcpy(&n, kv->c.err, sizeof n, hipMemcpyDeviceToHost));
    HIP_TRY(hipMemset(kv->c.err, 0, sizeof n));
    HIP_TRY(hipDeviceSynchronize());
    *n_invalid_slots = n;
    return LORA_OK;
}

int lora_attend_plan_create(int max_seqs, int max_groups, int max_tokens, int max_pages, int n_heads, int n_kv_heads,
                            int head_dim, lora_attend_plan *out) {
    if (out == nullptr) return LORA_EINVAL;
    *out = nullptr;
    if (max_seqs < 1 || max_groups < 0 || max_tokens < 1 || max_pages < 0 || !dim_ok(head_dim)) return LORA_EINVAL;
    if (max_seqs > LORA_ATTEND_MAX_TOKENS || max_groups > LORA_ATTEND_MAX_TOKENS ||
        max_tokens > LORA_ATTEND_MAX_TOKENS || max_pages > LORA_ATTEND_MAX_PAGES)
        return LORA_EINVAL;
    if (n_kv_heads < 1 || n_kv_heads > LORA_KV_MAX_HEADS || n_heads < n_kv_heads || n_heads % n_kv_heads != 0 ||
        n_heads / n_kv_heads > lora::ATTEND_MAX_GQ)
        return LORA_EINVAL;
    lora_attend_plan p = nullptr;
    try {
        p = new lora_attend_plan_s(max_seqs, max_groups, max_tokens, max_pages, n_heads, n_kv_heads);
    } catch (const std::exception &) {
        return LORA_ENOMEM;
    }
    p->max_tokens = max_tokens;
    p->n_heads = n_heads;
    p->n_kv_heads = n_kv_heads;
    p->head_dim = head_dim;
    const size_t plan_bytes = align_up(p->planner.max_bytes(), 256);
    const size_t rows = static_cast<size_t>(p->planner.max_part_rows()) * n_heads;
    const size_t o_bytes = align_up(rows * head_dim * 4, 256);
    const size_t ml_bytes = align_up(rows * 8, 256);
    const size_t cnt_bytes = static_cast<size_t>(max_tokens) * n_kv_heads * 4;
    hipError_t e = hipGetDevice(&p->device);
    if (e == hipSuccess)
        e = hipMalloc(reinterpret_cast<void **>(&p->mem), plan_bytes + o_bytes + ml_bytes + cnt_bytes);
    // The counters start at 0; every call leaves them there.
    if (e == hipSuccess) e = hipMemset(p->mem + plan_bytes + o_bytes + ml_bytes, 0, cnt_bytes);
    if (e == hipSuccess) e = hipDeviceSynchronize();
    for (int i = 0; i < 2; ++i) {
        if (e == hipSuccess) e = hipHostMalloc(&p->host[i], plan_bytes, hipHostMallocDefault);
        if (e == hipSuccess) e = hipEventCreateWithFlags(&p->sent[i], hipEventDisableTiming);
    }
    if (e != hipSuccess) {
        const int rc = alloc_status(e);
        free_plan(p);
        delete p;
        return rc;
    }
    p->part_o = reinterpret_cast<float *>(p->mem + plan_bytes);
    p->part_ml = reinterpret_cast<float *>(p->mem + plan_bytes + o_bytes);
    p->count = reinterpret_cast<unsigned *>(p->mem + plan_bytes + o_bytes + ml_bytes);
    *out = p;
    return LORA_OK;
}

int lora_attend_plan_destroy(lora_attend_plan plan) {
    if (plan == nullptr) return LORA_OK;
    int rc = LORA_OK;
    {
        DeviceGuard g(plan->device);
        const hipError_t e = g.error() == hipSuccess ? hipDeviceSynchronize() : g.error();
        if (e != hipSuccess) rc = hip_fail(e);
        free_plan(plan);
    }
    delete plan;
    return rc;
}

int lora_attend_plan_set(lora_attend_plan plan, lora_kv kv, const lora_attend_batch *batch, void *stream) {
    return set_plan(plan, kv, batch, nullptr, false, stream);
}

int lora_attend_plan_set_tree(lora_attend_plan plan, lora_kv kv, const lora_attend_batch *batch,
                              const int32_t *parent, void *stream) {
    return set_plan(plan, kv, batch, parent, true, stream);
}

int lora_attend(lora_kv kv, lora_attend_plan plan, const void *q, int64_t q_stride, float scale, void *out,
                float *lse, void *stream) {
    if (kv == nullptr || plan == nullptr || !std::isfinite(scale)) return LORA_EINVAL;
    std::lock_guard<std::mutex> lk(plan->mu);
    if (!plan->set) return LORA_EINVAL;
    if (kv->device != plan->device || kv->c.heads != plan->n_kv_heads || kv->c.dim != plan->head_dim ||
        kv->page_size != plan->page_size || kv->c.n_pages != plan->n_pages)
        return LORA_EMISMATCH;
    int n_tokens = static_cast<int>(plan->planner.tokens().size()), n_groups = plan->planner.groups();
    int join_steps = plan->planner.join_steps();
    DeviceGuard g(plan->device);
    HIP_TRY(g.error());
    if (n_tokens == 0) {
        // Nothing to do now, but a graph that captures the call may be
        // replayed after plans of any size: launched to fill the device.
        hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
        HIP_TRY(hipStreamIsCapturing(static_cast<hipStream_t>(stream), &cap));
        if (cap == hipStreamCaptureStatusNone) return LORA_OK;
        n_tokens = join_steps = plan->max_tokens;
        n_groups = (lora::ATTEND_SLOTS / lora::ATTEND_WAVES + plan->n_kv_heads - 1) / plan->n_kv_heads;
    }
    const int64_t row = static_cast<int64_t>(plan->n_heads) * plan->head_dim;
    if (q == nullptr || out == nullptr || q == out || q_stride < row || q_stride % 8 != 0) return LORA_EINVAL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return LORA_EINVAL;
    lora::AttendArgs a{};
    a.meta = plan->mem;
    a.k = kv->c.k;
    a.v = kv->c.v;
    a.kexp = kv->c.kexp;
    a.vinv = kv->c.vinv;
    a.q = static_cast<const uint16_t *>(q);
    a.q_stride = q_stride;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.part_o = plan->part_o;
    a.part_ml = plan->part_ml;
    a.count = plan->count;
    a.heads = plan->n_heads;
    a.kv_heads = plan->n_kv_heads;
    a.gq = plan->n_heads / plan->n_kv_heads;
    a.gq_inv = (65536 + a.gq - 1) / a.gq;
    a.page_shift = kv->c.page_shift;
    a.n_pages = kv->c.n_pages;
    a.scale = scale * 1.44269504088896340736f;
    HIP_TRY(lora::launch_attend(a, kv->c.dtype, plan->head_dim, n_groups, n_tokens, join_steps,
                                static_cast<hipStream_t>(stream)));
    return LORA_OK;
}

int lora_verifier_create(int max_seqs, lora_verifier *out) {
    if (out == nullptr) return LORA_EINVAL;
    *out = nullptr;
    if (max_seqs < 1 || max_seqs > LORA_VERIFY_MAX_SEQS) return LORA_EINVAL;
    lora_verifier v = new (std::nothrow) lora_verifier_s;
    if (v == nullptr) return LORA_ENOMEM;
    v->max_seqs = max_seqs;
    const size_t sums = static_cast<size_t>(max_seqs) * lora::VERIFY_PARTS * sizeof(double);
    const size_t count = align_up(static_cast<size_t>(max_seqs) * sizeof(unsigned), 256);
    const size_t row_sums = static_cast<size_t>(lora::VERIFY_TREE_ROWS) * lora::VERIFY_CHUNKS * sizeof(double);
    const size_t total = sums + count + row_sums + static_cast<size_t>(lora::VERIFY_TREE_ROWS) * sizeof(unsigned);
    hipError_t e = hipGetDevice(&v->device);
    if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void **>(&v->mem), total);
    if (e == hipSuccess) e = hipMemset(v->mem, 0, total);
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) {
        const int rc = alloc_status(e);
        if (v->mem) (void)hipFree(v->mem);
        delete v;
        return rc;
    }
    v->sums = reinterpret_cast<double *>(v->mem);
    v->count = reinterpret_cast<unsigned *>(v->mem + sums);
    v->row_sums = reinterpret_cast<double *>(v->mem + sums + count);
    v->row_count = reinterpret_cast<unsigned *>(v->mem + sums + count + row_sums);
    *out = v;
    return LORA_OK;
}

int lora_verifier_destroy(lora_verifier v) {
    if (v == nullptr) return LORA_OK;
    const int rc = free_on(v->device, v->mem);
    delete v;
    return rc;
}

int lora_verify(lora_verifier v, const void *p_target, const void *p_draft, lora_dtype dtype, int vocab,
                const int32_t *draft, const int32_t *row0, const float *u, int n_seqs, int n_rows, int32_t *tokens,
                int32_t *accepted, void *stream) {
    if (v == nullptr || n_seqs < 0 || n_rows < 0 || vocab < 1 || vocab > LORA_VERIFY_MAX_VOCAB) return LORA_EINVAL;
    if (dtype != LORA_F32 && dtype != LORA_F16 && dtype != LORA_BF16) return LORA_EINVAL;
    if (n_seqs == 0) return LORA_OK;
    if (n_seqs > v->max_seqs) return LORA_ETOKENS;
    // A sequence has one row more than drafted tokens, so n_rows <= n_seqs
    // leaves none: p_draft and draft are then not looked at.
    const size_t esz = dtype == LORA_F32 ? 4 : 2;
    if (row0 == nullptr || accepted == nullptr || !aligned(row0, 4) || !aligned(accepted, 4)) return LORA_EINVAL;
    if (n_rows > 0 && (p_target == nullptr || u == nullptr || tokens == nullptr)) return LORA_EINVAL;
    if (n_rows > n_seqs && (p_draft == nullptr || draft == nullptr)) return LORA_EINVAL;
    if (!aligned(p_target, esz) || !aligned(p_draft, esz) || !aligned(draft, 4) || !aligned(u, 4) ||
        !aligned(tokens, 4))
        return LORA_EINVAL;
    DeviceGuard g(v->device);
    HIP_TRY(g.error());
    lora::VerifyArgs a{};
    a.p = p_target;
    a.q = p_draft;
    a.draft = draft;
    a.row0 = row0;
    a.u = u;
    a.tokens = tokens;
    a.accepted = accepted;
    a.sums = v->sums;
    a.count = v->count;
    a.n_seqs = n_seqs;
    a.n_rows = n_rows;
    a.vocab = vocab;
    // A workgroup fills a CU: as many to a sequence as there are CUs for it.
    a.parts = (vocab + lora::VERIFY_PART - 1) / lora::VERIFY_PART;
    const int wgs = 256 / n_seqs;
    a.group = wgs < 1 ? a.parts : (a.parts + wgs - 1) / wgs;
    HIP_TRY(lora::launch_verify(a, static_cast<int>(dtype), static_cast<hipStream_t>(stream)));
    return LORA_OK;
}

int lora_verify_tree(lora_verifier v, const void *p_target, lora_dtype dtype, int vocab, const int32_t *draft,
                     const int32_t *parent, const int32_t *row0, const float *u, int n_seqs, int n_rows,
                     int32_t *tokens, int32_t *path, int32_t *accepted, void *stream) {
    if (v == nullptr || n_seqs < 0 || n_rows < 0 || vocab < 1 || vocab > LORA_VERIFY_MAX_VOCAB) return LORA_EINVAL;
    if (dtype != LORA_F32 && dtype != LORA_F16 && dtype != LORA_BF16) return LORA_EINVAL;
    if (n_seqs == 0) return LORA_OK;
    if (n_seqs > v->max_seqs) return LORA_ETOKENS;
    if (row0 == nullptr || accepted == nullptr || !aligned(row0, 4) || !aligned(accepted, 4)) return LORA_EINVAL;
    if (n_rows > 0 && (p_target == nullptr || draft == nullptr || parent == nullptr || u == nullptr ||
                       tokens == nullptr || path == nullptr))
        return LORA_EINVAL;
    if (!aligned(p_target, dtype == LORA_F32 ? 4 : 2) || !aligned(draft, 4) || !aligned(parent, 4) || !aligned(u, 4) ||
        !aligned(tokens, 4) || !aligned(path, 4))
        return LORA_EINVAL;
    DeviceGuard g(v->device);
    HIP_TRY(g.error());
    lora::VerifyTreeArgs a{};
    a.p = p_target;
    a.draft = draft;
    a.parent = parent;
    a.row0 = row0;
    a.u = u;
    a.tokens = tokens;
    a.path = path;
    a.accepted = accepted;
    a.n_seqs = n_seqs;
    a.n_rows = n_rows;
    a.vocab = vocab;
    a.sums = v->row_sums;
    a.count_row = v->row_count;
    a.count = v->count;
    HIP_TRY(lora::launch_verify_tree(a, static_cast<int>(dtype), static_cast<hipStream_t>(stream)));
    return LORA_OK;
}

int lora_scorer_create(int max_rows, lora_scorer *out) {
    if (out == nullptr) return LORA_EINVAL;
    *out = nullptr;
    if (max_rows < 1 || max_rows > LORA_SCORE_MAX_ROWS) return LORA_EINVAL;
    lora_scorer s = new (std::nothrow) lora_scorer_s;
    if (s == nullptr) return LORA_ENOMEM;
    s->max_rows = max_rows;
    const size_t keys = static_cast<size_t>(lora::LOGPROBS_WGS) * lora::LOGPROBS_MAX_TOP * sizeof(uint64_t);
    const size_t stats = static_cast<size_t>(lora::LOGPROBS_WGS) * 4 * sizeof(float);
    const size_t total = keys + stats + static_cast<size_t>(lora::LOGPROBS_WGS) * sizeof(unsigned);
    hipError_t e = hipGetDevice(&s->device);
    if (e == hipSuccess) e = hipMalloc(reinterpret_cast<void **>(&s->mem), total);
    if (e == hipSuccess) e = hipMemset(s->mem, 0, total);
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) {
        const int rc = alloc_status(e);
        if (s->mem) (void)hipFree(s->mem);
        delete s;
        return rc;
    }
    s->keys = reinterpret_cast<uint64_t *>(s->mem);
    s->stats = reinterpret_cast<float *>(s->mem + keys);
    s->count = reinterpret_cast<unsigned *>(s->mem + keys + stats);
    *out = s;
    return LORA_OK;
}

int lora_scorer_destroy(lora_scorer s) {
    if (s == nullptr) return LORA_OK;
    const int rc = free_on(s->device, s->mem);
    delete s;
    return rc;
}

int lora_logprobs(lora_scorer s, const void *logits, int64_t stride, lora_dtype dtype, int vocab,
                  const int32_t *tokens, float scale, int top, int n_rows, float *logprob, float *entropy,
                  int32_t *top_ids, float *top_logprobs, void *stream) {
    if (s == nullptr || n_rows < 0 || vocab < 1 || vocab > LORA_VERIFY_MAX_VOCAB || stride < vocab) return LORA_EINVAL;
    if (dtype != LORA_F32 && dtype != LORA_F16 && dtype != LORA_BF16) return LORA_EINVAL;
    if (!(scale >= 0x1p-64f && scale <= 0x1p64f) || top < 0 || top > LORA_SCORE_MAX_TOP || top > vocab)
        return LORA_EINVAL;
    if (n_rows == 0) return LORA_OK;
    if (n_rows > s->max_rows) return LORA_ETOKENS;
    if (logits == nullptr || !aligned(logits, dtype == LORA_F32 ? 4 : 2)) return LORA_EINVAL;
    if (top > 0 && (top_ids == nullptr || top_logprobs == nullptr)) return LORA_EINVAL;
    if (!aligned(tokens, 4) || !aligned(logprob, 4) || !aligned(entropy, 4)) return LORA_EINVAL;
    if (top > 0 && (!aligned(top_ids, 4) || !aligned(top_logprobs, 4))) return LORA_EINVAL;
    DeviceGuard g(s->device);
    HIP_TRY(g.error());
    lora::LogprobsArgs a{};
    a.z = logits;
    a.stride = stride;
    a.tokens = tokens;
    a.c = scale * 1.44269504088896340736f;
    a.n_rows = n_rows;
    a.vocab = vocab;
    a.top = top;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.keys = s->keys;
    a.stats = s->stats;
    a.count = s->count;
    HIP_TRY(lora::launch_logprobs(a, static_cast<int>(dtype), static_cast<hipStream_t>(stream)));
    return LORA_OK;
}

}  // extern "C"
