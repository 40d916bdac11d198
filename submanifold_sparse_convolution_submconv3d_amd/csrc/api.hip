// C ABI of the submconv library: argument validation, rulebook lifetime,
// kernel dispatch.  Every argument check here runs before any HIP call, so
// invalid calls fail without touching the device.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <chrono>
#include <mutex>
#include <unordered_map>
#include <vector>

#include "attention.h"
#include "common.h"
#include "headnorm.h"
#include "linear.h"

namespace sc {
int build_map(const int32_t *coords, submconv_rulebook *rb, hipStream_t stream);
int launch_forward(const void *feats, const void *w, const float *bias,
                   const submconv_rulebook *rb, void *out, int cin, int cout, int dtype, int flip,
                   int variant, hipStream_t s);
int input_order_table(const submconv_rulebook *rb, int32_t *out, hipStream_t s);
int64_t win_plan_ints(int64_t n);
int subdivide(const int32_t *coords, const void *feats, int64_t n, int c, int dtype,
              int32_t *out_coords, void *out_feats, hipStream_t s);
int space_to_depth(const int32_t *coords, const void *feats, int64_t n, int c, int dtype, int res,
                   int batch, int32_t *out_coords, void *out_feats, uint8_t *out_mask,
                   int64_t *out_m, hipStream_t s);
int depth_to_space(const int32_t *cc, const void *cf, const uint8_t *mask, int64_t m, int c,
                   int dtype, int32_t *out_coords, void *out_feats, int64_t *out_n, hipStream_t s);
int upsample_masked(const int32_t *coords, const void *feats, const uint8_t *mask, int64_t n, int c, int dtype,
                    int32_t *out_coords, void *out_feats, int64_t *out_n, hipStream_t s);
int upsample_masked_noalloc(const int32_t *coords, const void *feats, const uint8_t *mask, int64_t n, int c,
                            int dtype, int32_t *out_coords, void *out_feats, int64_t *out_n, hipStream_t s);
size_t noalloc_expand_bytes(int64_t m);
int downsample(const int32_t *coords, const void *feats, int64_t n, int c, int dtype, int res, int batch,
               int mean, int32_t *out_coords, void *out_feats, int64_t *out_m, hipStream_t s);
int classify_5d(const int64_t *shape, int hint, int *layout);
int weight_convert(const void *src, int layout, int cout, int cin, int dtype, int flip, void *dst, hipStream_t s);
int layer_norm(const void *x, int64_t ldx, int64_t n, int c, int dtype, const void *w, const void *b, int pdtype,
               float eps, void *y, int64_t ldy, float *stats, hipStream_t s);
size_t norm_bwd_workspace(int64_t n, int c, int dtype);
int layer_norm_backward(const void *gy, int64_t ldg, const void *x, int64_t ldx, int64_t n, int c, int dtype,
                        const float *stats, const void *w, int pdtype, void *dx, int64_t lddx, void *dw, void *db,
                        void *workspace, hipStream_t s);
int rotary(const void *x, int64_t x_row, int64_t x_head, const int32_t *pos, int64_t pos_row, const float *freqs,
           const int32_t *sections, int axes, int64_t n, int heads, int dim, int dtype, int split, int inverse,
           void *out, int64_t out_row, int64_t out_head, hipStream_t s);
size_t attention_workspace(const AttnArgs &A, int dtype);
int attention(const AttnArgs &A, int dtype, void *workspace, hipStream_t s);
size_t attention_backward_workspace(const AttnArgs &A, int dtype);
int attention_backward(AttnArgs A, int dtype, void *workspace, hipStream_t s);
size_t route_workspace(int64_t n, int experts, int k);
int route(const void *logits, int64_t ld, int64_t n, int experts, int k, int dtype, int normalize, int32_t *chosen,
          float *gates, int32_t *offsets, int32_t *rows, int32_t *slots, void *workspace, hipStream_t s);
int route_none(int32_t *offsets, int experts, hipStream_t s);
int route_backward(const float *grad, const void *logits, int64_t ld, int64_t n, int experts, int k, int dtype,
                   int normalize, const int32_t *chosen, const float *gates, void *out, int64_t out_ld, hipStream_t s);
int combine(const void *y, int64_t ldy, int64_t np, const int32_t *slots, const float *gates, int64_t n, int k, int c,
            int dtype, void *out, int64_t ldo, hipStream_t s);
int combine_backward(const void *g, int64_t ldg, const void *y, int64_t ldy, int64_t np, const int32_t *slots,
                     const int32_t *rows, const float *gates, int64_t n, int k, int c, int dtype, void *dy,
                     int64_t lddy, float *dgates, hipStream_t s);

static thread_local char g_err[512];

int fail(int status, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return status;
}

// Pinned host blocks of a host thread: the status read-back buffer and the status
// mailbox.  A thread's blocks go back to a process-wide list when the thread exits
// (no HIP call there: the runtime may already be shutting down) and are handed to the
// next thread that needs one, so short-lived threads do not pile up pinned memory.
namespace {
struct PinnedSet {
    DevStatus *pinned = nullptr;   // read-back buffer
    size_t pinned_bytes = 0;
    Mailbox *mb = nullptr;         // host address of the mailbox
    Mailbox *mb_dev = nullptr;     // its device address
    uint32_t seq = 0;              // the last sequence number used on it
};
std::mutex g_pinned_mu;
std::vector<PinnedSet> g_pinned_free;
struct PinnedHolder {
    PinnedSet p;
    PinnedHolder()
    {
        std::lock_guard<std::mutex> lk(g_pinned_mu);
        if (!g_pinned_free.empty()) {
            p = g_pinned_free.back();
            g_pinned_free.pop_back();
        }
    }
    ~PinnedHolder()
    {
        if (!p.pinned && !p.mb) return;
        std::lock_guard<std::mutex> lk(g_pinned_mu);
        g_pinned_free.push_back(p);
    }
};
thread_local PinnedHolder g_pin;
}  // namespace

int read_status_counts(const DevStatus *d, int64_t ncounts, DevStatus *h, uint64_t *sum, hipStream_t stream)
{
    const size_t bytes = sizeof(DevStatus) + (size_t)ncounts * 4;
    PinnedSet &ps = g_pin.p;
    if (ps.pinned_bytes < bytes) {  // grows to the largest read-back seen on this thread
        if (ps.pinned) (void)hipHostFree(ps.pinned);
        ps.pinned = nullptr;
        ps.pinned_bytes = 0;
        const size_t want = bytes < 4096 ? 4096 : bytes;
        SC_HIP(hipHostMalloc((void **)&ps.pinned, want, hipHostMallocDefault));
        ps.pinned_bytes = want;
    }
    SC_HIP(hipMemcpyAsync(ps.pinned, d, bytes, hipMemcpyDeviceToHost, stream));
    SC_HIP(hipStreamSynchronize(stream));
    *h = *ps.pinned;
    uint64_t t = 0;
    const uint32_t *c = (const uint32_t *)(ps.pinned + 1);
    for (int64_t i = 0; i < ncounts; ++i) t += c[i];
    if (sum) *sum = t;
    return SUBMCONV_OK;
}

int read_status(const DevStatus *d, DevStatus *h, hipStream_t stream)
{
    return read_status_counts(d, 0, h, nullptr, stream);
}

int mailbox_acquire(Mailbox **mb, uint32_t *seq)
{
    PinnedSet &ps = g_pin.p;
    if (!ps.mb) {
        // coherent: the device's stores reach host memory while the kernel runs; portable:
        // usable from every device
        Mailbox *h = nullptr;
        SC_HIP(hipHostMalloc((void **)&h, sizeof(Mailbox),
                             hipHostMallocCoherent | hipHostMallocMapped | hipHostMallocPortable));
        __atomic_store_n(&h->seq, 0u, __ATOMIC_RELAXED);
        void *dp = nullptr;
        if (hipHostGetDevicePointer(&dp, h, 0) != hipSuccess) {
            (void)hipHostFree(h);
            return fail(SUBMCONV_E_HIP, "hipHostGetDevicePointer failed for the status mailbox");
        }
        ps.mb = h;
        ps.mb_dev = (Mailbox *)dp;
        ps.seq = 0;
    }
    // the sequence goes on from the mailbox's last one (it may come from an exited thread),
    // so a stale post never matches; never 0, the initial value
    ps.seq = ps.seq + 1 ? ps.seq + 1 : 1;
    *mb = ps.mb_dev;
    *seq = ps.seq;
    return SUBMCONV_OK;
}

int mailbox_wait(Mailbox *mb_dev, uint32_t seq, DevStatus *h, hipStream_t stream)
{
    (void)mb_dev;
    Mailbox *mb = g_pin.p.mb;
    // poll for up to ~2 ms (a build of a few million voxels takes well under that); past
    // it, or if the post never comes (a failed launch), synchronise and check once more
    const auto t0 = std::chrono::steady_clock::now();
    bool seen = false;
    for (uint32_t it = 0;; ++it) {
        if (__atomic_load_n(&mb->seq, __ATOMIC_ACQUIRE) == seq) {
            seen = true;
            break;
        }
        if ((it & 255u) == 255u && std::chrono::steady_clock::now() - t0 > std::chrono::microseconds(2000)) break;
    }
    if (!seen) {
        SC_HIP(hipStreamSynchronize(stream));
        if (__atomic_load_n(&mb->seq, __ATOMIC_ACQUIRE) != seq)
            return fail(SUBMCONV_E_HIP, "the build's status was not posted");
    }
    *h = DevStatus{};
    h->flags = mb->flags;
    h->taps = mb->taps;
    h->count = mb->count;
    return SUBMCONV_OK;
}

// Device memory of the library (rulebooks and scratch) comes from a block cache.
// The driver's stream-ordered allocator costs tens to hundreds of microseconds of
// host time per call for large blocks, and a map build allocates and frees its
// scratch every time; so freed blocks are kept per device and handed out again for
// requests of up to their size and at least half of it.
//
// Ordering: a block freed while work queued on a stream may still use it carries an
// event recorded on that stream at the free.  Whoever takes the block next makes its
// own stream wait for that event (hipStreamWaitEvent), so a block can move between
// streams, and a stream destroyed meanwhile leaves no dangling ordering.  Blocks
// freed right after their stream was synchronised carry no event.  Blocks of the
// caller's stream are preferred, so the usual wait is on an event of the same stream.
// The cache holds at most g_cap bytes per device (submconv_set_cache_limit; 2 GiB by
// default); beyond that, freed blocks go back to the driver.  submconv_release_cache
// empties it.
namespace {
struct Cached {
    void *p;
    size_t bytes;
    int device;
    hipStream_t stream;  // where it was freed (preference only)
    hipEvent_t ev;       // completes when that stream's prior work is done; nullptr: idle
};
std::mutex g_cache_mu;
size_t g_cap = size_t(2) << 30;
std::unordered_map<void *, std::pair<size_t, int>> g_live;  // block -> (bytes, device)
std::vector<Cached> g_free;
std::vector<std::pair<int, hipEvent_t>> g_events;  // spare events, by device
size_t g_cached[64];

size_t size_class(size_t bytes)  // 8 classes per power of two: at most 12.5% slack
{
    bytes = (bytes + 255) & ~size_t(255);
    size_t top = 256;
    while (top < bytes) top <<= 1;
    const size_t step = top >= 2048 ? top / 16 : 128;
    return (bytes + step - 1) / step * step;
}

void put_event(int device, hipEvent_t ev)  // caller holds g_cache_mu
{
    if (ev) g_events.push_back({device, ev});
}

hipEvent_t get_event(int device)  // caller holds g_cache_mu; current device == device
{
    for (size_t i = 0; i < g_events.size(); ++i)
        if (g_events[i].first == device) {
            hipEvent_t ev = g_events[i].second;
            g_events[i] = g_events.back();
            g_events.pop_back();
            return ev;
        }
    hipEvent_t ev = nullptr;
    if (hipEventCreateWithFlags(&ev, hipEventDisableTiming) != hipSuccess) return nullptr;
    return ev;
}

// Return blocks to the driver once their last use has finished.  Caller holds g_cache_mu.
void release_cached(int device)
{
    int cur = -1;
    (void)hipGetDevice(&cur);
    for (size_t i = 0; i < g_free.size();) {
        Cached &b = g_free[i];
        if (device < 0 || b.device == device) {
            if (b.ev) (void)hipEventSynchronize(b.ev);
            if (b.device != cur && hipSetDevice(b.device) == hipSuccess) cur = b.device;
            (void)hipFreeAsync(b.p, nullptr);  // its last use has finished (event above)
            put_event(b.device, b.ev);
            if (b.device >= 0 && b.device < 64) g_cached[b.device] -= b.bytes;
            g_free[i] = g_free.back();
            g_free.pop_back();
        } else {
            ++i;
        }
    }
}
}  // namespace

int dev_alloc(void **p, size_t bytes, hipStream_t stream)
{
    *p = nullptr;
    bytes = size_class(bytes == 0 ? 256 : bytes);
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return fail(SUBMCONV_E_HIP, "hipGetDevice failed");
    {
        std::lock_guard<std::mutex> lock(g_cache_mu);
        size_t best = SIZE_MAX;
        for (size_t i = 0; i < g_free.size(); ++i) {
            const Cached &b = g_free[i];
            if (b.device != dev || b.bytes < bytes || b.bytes / 2 > bytes) continue;
            if (best == SIZE_MAX) { best = i; continue; }
            const Cached &c = g_free[best];
            const bool bs = b.stream == stream, cs = c.stream == stream;
            if ((bs && !cs) || (bs == cs && b.bytes < c.bytes)) best = i;
        }
        if (best != SIZE_MAX) {
            Cached b = g_free[best];
            if (b.ev && hipStreamWaitEvent(stream, b.ev, 0) != hipSuccess)
                return fail(SUBMCONV_E_HIP, "hipStreamWaitEvent failed");
            put_event(dev, b.ev);
            *p = b.p;
            g_live[*p] = {b.bytes, dev};
            if (dev < 64) g_cached[dev] -= b.bytes;
            g_free[best] = g_free.back();
            g_free.pop_back();
            return SUBMCONV_OK;
        }
    }
    hipError_t e = hipMallocAsync(p, bytes, stream);
    if (e == hipErrorOutOfMemory) {  // give the cached blocks back and try once more
        {
            std::lock_guard<std::mutex> lock(g_cache_mu);
            release_cached(dev);
        }
        e = hipMallocAsync(p, bytes, stream);
    }
    if (e != hipSuccess) {
        *p = nullptr;
        return fail(e == hipErrorOutOfMemory ? SUBMCONV_E_OOM : SUBMCONV_E_HIP,
                    "device allocation of %zu bytes: %s", bytes, hipGetErrorString(e));
    }
    std::lock_guard<std::mutex> lock(g_cache_mu);
    g_live[*p] = {bytes, dev};
    return SUBMCONV_OK;
}

static void dev_release(void *p, hipStream_t stream, bool idle)
{
    if (!p) return;
    std::lock_guard<std::mutex> lock(g_cache_mu);
    auto it = g_live.find(p);
    if (it == g_live.end()) {  // not from dev_alloc: hand it to the driver
        (void)hipFreeAsync(p, stream);
        return;
    }
    const size_t bytes = it->second.first;
    const int dev = it->second.second;
    g_live.erase(it);
    int cur = -1;
    if (dev >= 0 && dev < 64 && g_cached[dev] + bytes <= g_cap && hipGetDevice(&cur) == hipSuccess && cur == dev) {
        hipEvent_t ev = nullptr;
        if (!idle) {
            ev = get_event(dev);
            if (!ev || hipEventRecord(ev, stream) != hipSuccess) {
                put_event(dev, ev);
                (void)hipFreeAsync(p, stream);
                return;
            }
        }
        g_free.push_back({p, bytes, dev, stream, ev});
        g_cached[dev] += bytes;
    } else {
        (void)hipFreeAsync(p, stream);
    }
}

void dev_free(void *p, hipStream_t stream) { dev_release(p, stream, false); }

void dev_free_idle(void *p, hipStream_t stream) { dev_release(p, stream, true); }

static bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

static bool overlaps(const void *a, size_t na, const void *b, size_t nb)
{
    const char *x = (const char *)a, *y = (const char *)b;
    return x < y + nb && y < x + na;
}

static size_t elem_size(int dtype) { return dtype == SUBMCONV_F32 ? 4 : 2; }

static bool known_dtype(int dtype) { return dtype == SUBMCONV_F32 || dtype == SUBMCONV_BF16; }
static bool aligned_to(const void *p, size_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

// Rows of the strided tensors: their number, and the largest distance in elements, such
// that every byte offset below fits 63 bits.
constexpr int64_t MAX_ROWS = int64_t(1) << 31, MAX_STRIDE = int64_t(1) << 24;

// Memory a call reads or writes: n x heads pieces of `dim` bytes, rows `row` bytes apart
// and heads `head` bytes apart (one piece: n = heads = 1).
struct Range {
    const char *what;
    const void *p;
    bool written;
    int64_t n, row, heads, head, dim;

    int64_t bytes() const { return p && n > 0 && dim > 0 ? (n - 1) * row + (heads - 1) * head + dim : 0; }
};

static Range range1(const char *what, const void *p, size_t bytes, bool written) { return Range{what, p, written, 1, 0, 1, 0, (int64_t)bytes}; }

static Range range2(const char *what, const void *p, int64_t n, int64_t c, int64_t ld, size_t es, bool written)
{
    return Range{what, p, written, n, ld * (int64_t)es, 1, 0, c * (int64_t)es};
}

// Whether two ranges share bytes; exact where their rows and heads are equally far apart, as
// parts of one wider tensor are, else by whole rows, whole heads or the whole span.
static bool collide(Range a, Range b)
{
    if (!a.bytes() || !b.bytes() || !overlaps(a.p, a.bytes(), b.p, b.bytes())) return false;
    // a distance that is not used is as good as any
    if (a.n == 1) a.row = b.row;
    if (b.n == 1) b.row = a.row;
    if (a.heads == 1) a.head = b.head;
    if (b.heads == 1) b.head = a.head;
    if (a.row != b.row && a.head != b.head) return true;
    for (Range *r : {&a, &b}) {
        if (a.head != b.head) r->dim += (r->heads - 1) * r->head, r->heads = 1;
        else if (a.row != b.row) r->dim += (r->n - 1) * r->row, r->n = 1;
    }
    // Two pieces i and h steps apart lie at d - i row - h head of each other, and share bytes
    // where that is between -b.dim and a.dim.  For every h, the first i below the upper end:
    const int64_t d = (int64_t)((intptr_t)b.p - (intptr_t)a.p);
    const int64_t row = a.n > 1 ? a.row : b.row, head = a.heads > 1 ? a.head : b.head;
    for (int64_t h = 1 - b.heads; h < a.heads; ++h) {
        const int64_t e = d - h * head, over = e - a.dim;
        int64_t i = 1 - b.n;
        if (row > 0) {
            const int64_t first = (over >= 0 ? over / row : -((-over + row - 1) / row)) + 1;
            if (first > i) i = first;
        }
        if (i < a.n && e - i * row < a.dim && e - i * row > -b.dim) return true;
    }
    return false;
}

// A written range may share bytes with no other.
static int ranges_check(const Range *r, int n)
{
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && r[i].written && !(r[j].written && j < i) && collide(r[i], r[j]))
                return fail(SUBMCONV_E_ALIAS, "%s overlaps %s", r[i].what, r[j].what);
    return SUBMCONV_OK;
}

}  // namespace sc

using namespace sc;

extern "C" {

const char *submconv_version(void) { return "submconv 0.1 gfx950"; }

const char *submconv_status_string(int status)
{
    switch (status) {
    case SUBMCONV_OK: return "ok";
    case SUBMCONV_E_INVALID_ARG: return "invalid argument";
    case SUBMCONV_E_COORD_RANGE: return "coordinate out of range";
    case SUBMCONV_E_DUPLICATE: return "duplicate coordinate";
    case SUBMCONV_E_UNSUPPORTED: return "unsupported configuration";
    case SUBMCONV_E_ALIAS: return "output aliases an input";
    case SUBMCONV_E_OOM: return "out of device memory";
    case SUBMCONV_E_HIP: return "HIP runtime error";
    }
    return "unknown status";
}

const char *submconv_last_error(void) { return g_err; }

int submconv_build_map(const int32_t *coords, int64_t n, int32_t res, int32_t batch, void *stream,
                       submconv_rulebook **out_rb)
{
    if (!out_rb) return fail(SUBMCONV_E_INVALID_ARG, "out_rb is NULL");
    *out_rb = nullptr;
    if (n < 0 || n >= (int64_t(1) << 31)) return fail(SUBMCONV_E_INVALID_ARG, "n = %lld outside [0, 2^31)", (long long)n);
    if (n > 0 && !coords) return fail(SUBMCONV_E_INVALID_ARG, "coords is NULL");
    if (n > 0 && !aligned16(coords)) return fail(SUBMCONV_E_INVALID_ARG, "coords must be 16-byte aligned");
    if (res < 1) return fail(SUBMCONV_E_INVALID_ARG, "res = %d must be >= 1", res);
    if (batch < 1) return fail(SUBMCONV_E_INVALID_ARG, "batch = %d must be >= 1", batch);
    const int rb = bits_for(res) > 0 ? bits_for(res) : 1;
    const int nbits = 3 * rb + bits_for(batch);
    if (nbits > 64) return fail(SUBMCONV_E_UNSUPPORTED, "res %d and batch %d need %d key bits (max 64)", res, batch, nbits);
    hipStream_t s = (hipStream_t)stream;

    submconv_rulebook *r = new (std::nothrow) submconv_rulebook();
    if (!r) return fail(SUBMCONV_E_OOM, "host allocation failed");
    r->n = n;
    r->res = res;
    r->batch = batch;
    r->rb = rb;
    r->nbits = nbits;
    r->key_bytes = nbits <= 32 ? 4 : 8;
    r->taps = 0;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) { delete r; return fail(SUBMCONV_E_HIP, "hipGetDevice failed"); }
    r->device = dev;
    int st = SUBMCONV_OK;
    r->ngroups = (n + 31) / 32;
    r->nbr_in = nullptr;

    const size_t kbytes = (((size_t)n * r->key_bytes) + 255) & ~size_t(255);
    const size_t pbytes = (((size_t)n * 4) + 255) & ~size_t(255);
    // +1 KB: kernels copy table rows in 16-byte chunks that may run past the last row
    const size_t nbytes = ((((size_t)n * NBR_INTS * 4) + 255) & ~size_t(255)) + 1024;
    const size_t mbytes = (((size_t)r->ngroups * GWIN_INTS * 4) + 255) & ~size_t(255);
    const size_t lbytes = (size_t)win_plan_ints(n) * 4 + 256;
    r->block_bytes = kbytes + pbytes + nbytes + mbytes + lbytes;
    st = dev_alloc(&r->block, r->block_bytes, s);
    if (st != SUBMCONV_OK) { delete r; return st; }
    r->keys = r->block;
    r->perm = (int32_t *)((char *)r->block + kbytes);
    r->nbr_sp = (int32_t *)((char *)r->block + kbytes + pbytes);
    r->gwin = (int32_t *)((char *)r->block + kbytes + pbytes + nbytes);
    r->plan = (int32_t *)((char *)r->block + kbytes + pbytes + nbytes + mbytes);
    if (n > 0) {
        st = build_map(coords, r, s);
        if (st != SUBMCONV_OK) {
            dev_free(r->block, s);
            delete r;
            return st;
        }
    }
    *out_rb = r;
    return SUBMCONV_OK;
}

int submconv_rulebook_neighbors(submconv_rulebook *rb, void *stream, const int32_t **nbr, int64_t *n)
{
    if (!rb || !nbr || !n) return fail(SUBMCONV_E_INVALID_ARG, "NULL argument");
    if (!rb->nbr_in && rb->n > 0) {
        void *p = nullptr;
        SC_CHECK(dev_alloc(&p, (size_t)rb->n * 27 * 4, (hipStream_t)stream));
        const int st = input_order_table(rb, (int32_t *)p, (hipStream_t)stream);
        if (st != SUBMCONV_OK) { dev_free(p, (hipStream_t)stream); return st; }
        rb->nbr_in = (int32_t *)p;
    }
    *nbr = rb->nbr_in;
    *n = rb->n;
    return SUBMCONV_OK;
}

int submconv_rulebook_copy_neighbors(const submconv_rulebook *rb, int32_t *dst, void *stream)
{
    if (!rb) return fail(SUBMCONV_E_INVALID_ARG, "rulebook is NULL");
    if (rb->n == 0) return SUBMCONV_OK;
    if (!dst) return fail(SUBMCONV_E_INVALID_ARG, "dst is NULL");
    const size_t bytes = (size_t)rb->n * 27 * 4;
    if (overlaps(dst, bytes, rb->block, rb->block_bytes)) return fail(SUBMCONV_E_ALIAS, "dst overlaps the rulebook");
    return input_order_table(rb, dst, (hipStream_t)stream);
}

int submconv_rulebook_info(const submconv_rulebook *rb, int64_t *n, int32_t *res, int32_t *batch,
                           int64_t *taps_present)
{
    if (!rb) return fail(SUBMCONV_E_INVALID_ARG, "rulebook is NULL");
    if (n) *n = rb->n;
    if (res) *res = rb->res;
    if (batch) *batch = rb->batch;
    if (taps_present) *taps_present = rb->taps;
    return SUBMCONV_OK;
}

int submconv_rulebook_free(submconv_rulebook *rb, void *stream)
{
    if (!rb) return SUBMCONV_OK;
    dev_free(rb->nbr_in, (hipStream_t)stream);
    dev_free(rb->block, (hipStream_t)stream);
    delete rb;
    return SUBMCONV_OK;
}

int submconv_forward_variant(const void *feats, const void *weight, const float *bias,
                             const submconv_rulebook *rb, void *out, int32_t cin, int32_t cout,
                             int32_t dtype, int32_t flip, int32_t variant, void *stream)
{
    if (!rb) return fail(SUBMCONV_E_INVALID_ARG, "rulebook is NULL");
    if (dtype != SUBMCONV_F32 && dtype != SUBMCONV_BF16) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (cin < 1 || cin > 1024 || cout < 1 || cout > 1024)
        return fail(SUBMCONV_E_UNSUPPORTED, "channel counts %d -> %d outside 1..1024", cin, cout);
    if (flip != 0 && flip != 1) return fail(SUBMCONV_E_INVALID_ARG, "flip must be 0 or 1");
    if (variant < SUBMCONV_KERNEL_AUTO || variant > SUBMCONV_KERNEL_PERSISTENT)
        return fail(SUBMCONV_E_INVALID_ARG, "unknown kernel variant %d", variant);
    const int64_t n = rb->n;
    if (n == 0) return SUBMCONV_OK;
    if (!feats || !weight || !out) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    if (!aligned16(feats) || !aligned16(weight) || !aligned16(out) || (bias && !aligned16(bias)))
        return fail(SUBMCONV_E_INVALID_ARG, "tensor pointers must be 16-byte aligned");
    const size_t es = elem_size(dtype);
    const size_t fb = (size_t)n * cin * es, wb = (size_t)cout * 27 * cin * es, ob = (size_t)n * cout * es;
    if (overlaps(out, ob, feats, fb) || overlaps(out, ob, weight, wb) ||
        (bias && overlaps(out, ob, bias, (size_t)cout * 4)))
        return fail(SUBMCONV_E_ALIAS, "out overlaps feats, weight or bias");
    int dev = 0;
    if (hipGetDevice(&dev) == hipSuccess && dev != rb->device)
        return fail(SUBMCONV_E_INVALID_ARG, "rulebook lives on device %d, current device is %d", rb->device, dev);
    return launch_forward(feats, weight, bias, rb, out, cin, cout, dtype, flip, variant,
                          (hipStream_t)stream);
}

int submconv_forward(const void *feats, const void *weight, const float *bias,
                     const submconv_rulebook *rb, void *out, int32_t cin, int32_t cout,
                     int32_t dtype, int32_t flip, void *stream)
{
    return submconv_forward_variant(feats, weight, bias, rb, out, cin, cout, dtype, flip,
                                    SUBMCONV_KERNEL_AUTO, stream);
}

int submconv_subdivide(const int32_t *coords, const void *feats, int64_t n, int32_t c,
                       int32_t dtype, int32_t *out_coords, void *out_feats, void *stream)
{
    if (n < 0 || n >= (int64_t(1) << 28)) return fail(SUBMCONV_E_INVALID_ARG, "n = %lld outside [0, 2^28)", (long long)n);
    if (n == 0) return SUBMCONV_OK;
    if (!coords || !out_coords) return fail(SUBMCONV_E_INVALID_ARG, "NULL coordinate pointer");
    if (!aligned16(coords) || !aligned16(out_coords)) return fail(SUBMCONV_E_INVALID_ARG, "coordinate pointers must be 16-byte aligned");
    if (overlaps(out_coords, (size_t)n * 128, coords, (size_t)n * 16)) return fail(SUBMCONV_E_ALIAS, "out_coords overlaps coords");
    if (feats) {
        if (dtype != SUBMCONV_F32 && dtype != SUBMCONV_BF16) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
        if (c < 1 || c > 65536) return fail(SUBMCONV_E_INVALID_ARG, "c = %d", c);
        if (!out_feats) return fail(SUBMCONV_E_INVALID_ARG, "out_feats is NULL");
        const size_t es = elem_size(dtype);
        if (((uintptr_t)feats | (uintptr_t)out_feats) & (((size_t)c * es) % 4 == 0 ? 3u : 1u))
            return fail(SUBMCONV_E_INVALID_ARG, "feature pointers misaligned");
        if (overlaps(out_feats, (size_t)n * 8 * c * es, feats, (size_t)n * c * es))
            return fail(SUBMCONV_E_ALIAS, "out_feats overlaps feats");
    }
    return subdivide(coords, feats, n, c, dtype, out_coords, out_feats, (hipStream_t)stream);
}

int submconv_space_to_depth(const int32_t *coords, const void *feats, int64_t n, int32_t c,
                            int32_t dtype, int32_t res, int32_t batch, int32_t *out_coords,
                            void *out_feats, uint8_t *out_mask, int64_t *out_m, void *stream)
{
    if (!out_m) return fail(SUBMCONV_E_INVALID_ARG, "out_m is NULL");
    *out_m = 0;
    if (n < 0 || n >= (int64_t(1) << 31)) return fail(SUBMCONV_E_INVALID_ARG, "n = %lld outside [0, 2^31)", (long long)n);
    if (dtype != SUBMCONV_F32 && dtype != SUBMCONV_BF16) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (c < 1 || c > 65536) return fail(SUBMCONV_E_INVALID_ARG, "c = %d", c);
    if (res < 1 || batch < 1) return fail(SUBMCONV_E_INVALID_ARG, "res and batch must be >= 1");
    if (n == 0) return SUBMCONV_OK;
    if (!coords || !feats || !out_coords || !out_feats) return fail(SUBMCONV_E_INVALID_ARG, "NULL pointer");
    if (!aligned16(coords) || !aligned16(out_coords)) return fail(SUBMCONV_E_INVALID_ARG, "coordinate pointers must be 16-byte aligned");
    const size_t es = elem_size(dtype);
    if (overlaps(out_feats, (size_t)n * 8 * c * es, feats, (size_t)n * c * es) ||
        overlaps(out_coords, (size_t)n * 16, coords, (size_t)n * 16))
        return fail(SUBMCONV_E_ALIAS, "an output overlaps an input");
    return space_to_depth(coords, feats, n, c, dtype, res, batch, out_coords, out_feats, out_mask,
                          out_m, (hipStream_t)stream);
}

int submconv_depth_to_space(const int32_t *coarse_coords, const void *coarse_feats,
                            const uint8_t *mask, int64_t m, int32_t c, int32_t dtype,
                            int32_t *out_coords, void *out_feats, int64_t *out_n, void *stream)
{
    if (!out_n) return fail(SUBMCONV_E_INVALID_ARG, "out_n is NULL");
    *out_n = 0;
    if (m < 0 || m >= (int64_t(1) << 28)) return fail(SUBMCONV_E_INVALID_ARG, "m = %lld outside [0, 2^28)", (long long)m);
    if (dtype != SUBMCONV_F32 && dtype != SUBMCONV_BF16) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (c < 1 || c > 65536) return fail(SUBMCONV_E_INVALID_ARG, "c = %d", c);
    if (m == 0) return SUBMCONV_OK;
    if (!coarse_coords || !coarse_feats || !out_coords || !out_feats) return fail(SUBMCONV_E_INVALID_ARG, "NULL pointer");
    if (!aligned16(coarse_coords) || !aligned16(out_coords)) return fail(SUBMCONV_E_INVALID_ARG, "coordinate pointers must be 16-byte aligned");
    const size_t es = elem_size(dtype);
    if (overlaps(out_feats, (size_t)m * 8 * c * es, coarse_feats, (size_t)m * 8 * c * es) ||
        overlaps(out_coords, (size_t)m * 128, coarse_coords, (size_t)m * 16))
        return fail(SUBMCONV_E_ALIAS, "an output overlaps an input");
    return depth_to_space(coarse_coords, coarse_feats, mask, m, c, dtype, out_coords, out_feats,
                          out_n, (hipStream_t)stream);
}

static int check_upsample_masked(const int32_t *coords, const void *feats, const uint8_t *mask, int64_t n,
                                 int32_t c, int32_t dtype, int32_t *out_coords, void *out_feats, int64_t *out_n,
                                 int64_t max_n)
{
    if (!out_n) return fail(SUBMCONV_E_INVALID_ARG, "out_n is NULL");
    *out_n = 0;
    if (n < 0 || n >= (int64_t(1) << 28)) return fail(SUBMCONV_E_INVALID_ARG, "n = %lld outside [0, 2^28)", (long long)n);
    if (n > max_n) return fail(SUBMCONV_E_UNSUPPORTED, "n = %lld above the limit %lld", (long long)n, (long long)max_n);
    if (dtype != SUBMCONV_F32 && dtype != SUBMCONV_BF16) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (c < 1 || c > 65536) return fail(SUBMCONV_E_INVALID_ARG, "c = %d", c);
    if (n == 0) return SUBMCONV_OK;
    if (!coords || !feats || !mask || !out_coords || !out_feats) return fail(SUBMCONV_E_INVALID_ARG, "NULL pointer");
    if (!aligned16(coords) || !aligned16(out_coords)) return fail(SUBMCONV_E_INVALID_ARG, "coordinate pointers must be 16-byte aligned");
    const size_t es = elem_size(dtype);
    if (overlaps(out_feats, (size_t)n * 8 * c * es, feats, (size_t)n * c * es) ||
        overlaps(out_coords, (size_t)n * 128, coords, (size_t)n * 16) ||
        overlaps(out_feats, (size_t)n * 8 * c * es, mask, (size_t)n * 8) ||
        overlaps(out_coords, (size_t)n * 128, mask, (size_t)n * 8))
        return fail(SUBMCONV_E_ALIAS, "an output overlaps an input");
    return SUBMCONV_OK;
}

int submconv_upsample_masked(const int32_t *coords, const void *feats, const uint8_t *mask, int64_t n, int32_t c,
                             int32_t dtype, int32_t *out_coords, void *out_feats, int64_t *out_n, void *stream)
{
    SC_CHECK(check_upsample_masked(coords, feats, mask, n, c, dtype, out_coords, out_feats, out_n, int64_t(1) << 28));
    if (n == 0) return SUBMCONV_OK;
    return upsample_masked(coords, feats, mask, n, c, dtype, out_coords, out_feats, out_n, (hipStream_t)stream);
}

int submconv_upsample_masked_noalloc(const int32_t *coords, const void *feats, const uint8_t *mask, int64_t n,
                                     int32_t c, int32_t dtype, int32_t *out_coords, void *out_feats,
                                     int64_t *out_n, void *stream)
{
    static_assert(SUBMCONV_NOALLOC_MAX_N >= 1, "limit");
    SC_CHECK(check_upsample_masked(coords, feats, mask, n, c, dtype, out_coords, out_feats, out_n,
                                   SUBMCONV_NOALLOC_MAX_N));
    if (n == 0) return SUBMCONV_OK;
    if (noalloc_expand_bytes(n) > SUBMCONV_NOALLOC_SCRATCH_BYTES)  // cannot happen for n <= the limit
        return fail(SUBMCONV_E_UNSUPPORTED, "n = %lld does not fit the scratch array", (long long)n);
    return upsample_masked_noalloc(coords, feats, mask, n, c, dtype, out_coords, out_feats, out_n,
                                   (hipStream_t)stream);
}

int submconv_downsample(const int32_t *coords, const void *feats, int64_t n, int32_t c, int32_t dtype, int32_t res,
                        int32_t batch, int32_t mode, int32_t *out_coords, void *out_feats, int64_t *out_m,
                        void *stream)
{
    if (!out_m) return fail(SUBMCONV_E_INVALID_ARG, "out_m is NULL");
    *out_m = 0;
    if (n < 0 || n >= (int64_t(1) << 31)) return fail(SUBMCONV_E_INVALID_ARG, "n = %lld outside [0, 2^31)", (long long)n);
    if (dtype != SUBMCONV_F32 && dtype != SUBMCONV_BF16) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (mode != SUBMCONV_POOL_MAX && mode != SUBMCONV_POOL_MEAN) return fail(SUBMCONV_E_INVALID_ARG, "mode %d", mode);
    if (c < 1 || c > 65536) return fail(SUBMCONV_E_INVALID_ARG, "c = %d", c);
    if (res < 1 || batch < 1) return fail(SUBMCONV_E_INVALID_ARG, "res and batch must be >= 1");
    if (n == 0) return SUBMCONV_OK;
    if (!coords || !feats || !out_coords || !out_feats) return fail(SUBMCONV_E_INVALID_ARG, "NULL pointer");
    if (!aligned16(coords) || !aligned16(out_coords)) return fail(SUBMCONV_E_INVALID_ARG, "coordinate pointers must be 16-byte aligned");
    const size_t es = elem_size(dtype);
    if (overlaps(out_feats, (size_t)n * c * es, feats, (size_t)n * c * es) ||
        overlaps(out_coords, (size_t)n * 16, coords, (size_t)n * 16))
        return fail(SUBMCONV_E_ALIAS, "an output overlaps an input");
    return downsample(coords, feats, n, c, dtype, res, batch, mode == SUBMCONV_POOL_MEAN, out_coords, out_feats,
                      out_m, (hipStream_t)stream);
}

int submconv_classify_5d(const int64_t *shape, int32_t hint, int32_t *layout)
{
    if (!shape || !layout) return fail(SUBMCONV_E_INVALID_ARG, "NULL pointer");
    int l = SUBMCONV_LAYOUT_UNKNOWN;
    const int status = classify_5d(shape, hint, &l);
    *layout = l;
    return status;
}

int submconv_weight_convert(const void *src, int32_t layout, int32_t cout, int32_t cin, int32_t dtype, int32_t flip,
                            void *dst, void *stream)
{
    if (layout != SUBMCONV_LAYOUT_KRSC && layout != SUBMCONV_LAYOUT_OIDHW)
        return fail(SUBMCONV_E_INVALID_ARG, "layout %d", layout);
    if (dtype != SUBMCONV_F32 && dtype != SUBMCONV_BF16) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (cout < 1 || cin < 1 || (int64_t)cout * cin > (int64_t(1) << 24))
        return fail(SUBMCONV_E_INVALID_ARG, "cout = %d, cin = %d", cout, cin);
    if (!src || !dst) return fail(SUBMCONV_E_INVALID_ARG, "NULL pointer");
    const size_t bytes = (size_t)cout * 27 * cin * elem_size(dtype);
    if (overlaps(dst, bytes, src, bytes)) return fail(SUBMCONV_E_ALIAS, "dst overlaps src");
    return weight_convert(src, layout, cout, cin, dtype, flip, dst, (hipStream_t)stream);
}

static int norm_check(int64_t n, int32_t c, int32_t dtype, int32_t pdtype)
{
    if (n < 0 || n >= MAX_ROWS) return fail(SUBMCONV_E_INVALID_ARG, "n = %lld outside [0, 2^31)", (long long)n);
    if (!known_dtype(dtype) || !known_dtype(pdtype)) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d, param_dtype %d", dtype, pdtype);
    if (c < 1 || c > SUBMCONV_NORM_MAX_C)
        return fail(SUBMCONV_E_UNSUPPORTED, "c = %d outside 1..%d", c, SUBMCONV_NORM_MAX_C);
    return SUBMCONV_OK;
}

// Rows of an input may overlap or be one row (distance 0), those of an output may not.
static int row_check(const char *what, int64_t ld, int32_t least)
{
    if (ld < least || ld > MAX_STRIDE)
        return fail(SUBMCONV_E_INVALID_ARG, "%s rows are %lld elements apart, outside [%d, 2^24]", what, (long long)ld, least);
    return SUBMCONV_OK;
}

int submconv_layer_norm(const void *x, int64_t x_row, int64_t n, int32_t c, int32_t dtype, const void *weight,
                        const void *bias, int32_t param_dtype, float eps, void *y, int64_t y_row, float *stats,
                        void *stream)
{
    SC_CHECK(norm_check(n, c, dtype, param_dtype));
    SC_CHECK(row_check("x", x_row, 0));
    SC_CHECK(row_check("y", y_row, c));
    if (!(eps >= 0.0f)) return fail(SUBMCONV_E_INVALID_ARG, "eps = %g", (double)eps);
    if (n == 0) return SUBMCONV_OK;
    if (!x || !y) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
    if (!aligned_to(x, es) || !aligned_to(y, es) || !aligned_to(weight, ps) || !aligned_to(bias, ps) || !aligned_to(stats, 8))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    // y in the place of x is fine
    const Range r[] = {range2("x", x == y && (x_row == y_row || n == 1) ? nullptr : x, n, c, x_row, es, false),
                       range2("y", y, n, c, y_row, es, true), range1("weight", weight, (size_t)c * ps, false),
                       range1("bias", bias, (size_t)c * ps, false), range1("stats", stats, (size_t)n * 8, true)};
    SC_CHECK(ranges_check(r, 5));
    return layer_norm(x, x_row, n, c, dtype, weight, bias, param_dtype, eps, y, y_row, stats, (hipStream_t)stream);
}

size_t submconv_layer_norm_backward_workspace(int64_t n, int32_t c, int32_t dtype)
{
    return norm_check(n, c, dtype, SUBMCONV_F32) == SUBMCONV_OK ? norm_bwd_workspace(n, c, dtype) : 0;
}

int submconv_layer_norm_backward(const void *grad, int64_t grad_row, const void *x, int64_t x_row, int64_t n,
                                 int32_t c, int32_t dtype, const float *stats, const void *weight,
                                 int32_t param_dtype, void *dx, int64_t dx_row, void *dweight, void *dbias,
                                 void *workspace, size_t workspace_bytes, void *stream)
{
    SC_CHECK(norm_check(n, c, dtype, param_dtype));
    SC_CHECK(row_check("grad", grad_row, 0));
    SC_CHECK(row_check("x", x_row, 0));
    SC_CHECK(row_check("dx", dx_row, c));
    if (n && (!grad || !x || !stats || !dx)) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
    if (!aligned_to(grad, es) || !aligned_to(x, es) || !aligned_to(dx, es) || !aligned_to(stats, 8) ||
        !aligned_to(weight, ps) || !aligned_to(dweight, ps) || !aligned_to(dbias, ps) || !aligned16(workspace))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const size_t need = dweight || dbias ? norm_bwd_workspace(n, c, dtype) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return fail(SUBMCONV_E_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    const size_t pb = (size_t)c * ps;
    // dx in the place of grad is fine
    const Range r[] = {range2("grad", grad == dx && (grad_row == dx_row || n == 1) ? nullptr : grad, n, c, grad_row, es, false),
                       range2("x", x, n, c, x_row, es, false), range2("dx", dx, n, c, dx_row, es, true),
                       range1("stats", stats, (size_t)n * 8, false), range1("weight", weight, pb, false),
                       range1("dweight", dweight, pb, true), range1("dbias", dbias, pb, true),
                       range1("workspace", workspace, need, true)};
    SC_CHECK(ranges_check(r, 8));
    return layer_norm_backward(grad, grad_row, x, x_row, n, c, dtype, stats, weight, param_dtype, dx, dx_row, dweight,
                               dbias, workspace, (hipStream_t)stream);
}

// [n, heads, dim] with the given element distances.
static Range range3(const char *what, const void *p, int64_t n, int64_t heads, int64_t dim, int64_t row, int64_t head,
                    size_t es, bool written)
{
    const int64_t b = (int64_t)es;
    return Range{what, p, written, n, row * b, heads, head * b, dim * b};
}

// The distances of an [n, heads, dim] tensor; one that is written has each element once.
static int heads_check(const char *what, int64_t n, int64_t heads, int64_t dim, int64_t row, int64_t head, bool written)
{
    if (row < 0 || head < 0 || row > MAX_STRIDE || head > int64_t(1) << 40)
        return fail(SUBMCONV_E_INVALID_ARG, "%s: row distance %lld outside [0, 2^24] or head distance %lld outside [0, 2^40]",
                    what, (long long)row, (long long)head);
    const bool by_row = (heads <= 1 || head >= dim) && (n <= 1 || row >= (heads - 1) * head + dim);
    const bool by_head = (n <= 1 || row >= dim) && (heads <= 1 || head >= (n - 1) * row + dim);
    if (written && !by_row && !by_head)
        return fail(SUBMCONV_E_INVALID_ARG, "%s: heads or rows overlap (distances %lld, %lld)", what, (long long)row,
                    (long long)head);
    return SUBMCONV_OK;
}

int submconv_rotary(const void *x, int64_t x_row, int64_t x_head, const int32_t *positions, int64_t pos_row,
                    const float *freqs, const int32_t *sections, int32_t axes, int64_t n, int32_t heads, int32_t dim,
                    int32_t dtype, int32_t split, int32_t inverse, void *out, int64_t out_row, int64_t out_head,
                    void *stream)
{
    if (n < 0 || n >= MAX_ROWS) return fail(SUBMCONV_E_INVALID_ARG, "n = %lld outside [0, 2^31)", (long long)n);
    if (!known_dtype(dtype)) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (dim < 2 || dim > 512 || dim % 2) return fail(SUBMCONV_E_UNSUPPORTED, "dim = %d is not an even number in 2..512", dim);
    if (heads < 1 || heads > 1024) return fail(SUBMCONV_E_UNSUPPORTED, "heads = %d outside 1..1024", heads);
    if (axes < 1 || axes > SUBMCONV_ROTARY_MAX_AXES)
        return fail(SUBMCONV_E_UNSUPPORTED, "axes = %d outside 1..%d", axes, SUBMCONV_ROTARY_MAX_AXES);
    if ((split | inverse) & ~1) return fail(SUBMCONV_E_INVALID_ARG, "split and inverse must be 0 or 1");
    if (!sections) return fail(SUBMCONV_E_INVALID_ARG, "sections is NULL");
    int64_t pairs = 0;
    for (int a = 0; a < axes; ++a) {
        if (sections[a] < 0) return fail(SUBMCONV_E_INVALID_ARG, "sections[%d] = %d", a, sections[a]);
        pairs += sections[a];
    }
    if (pairs > dim / 2) return fail(SUBMCONV_E_INVALID_ARG, "sections hold %lld pairs, a head has %d", (long long)pairs, dim / 2);
    SC_CHECK(heads_check("x", n, heads, dim, x_row, x_head, false));
    SC_CHECK(heads_check("out", n, heads, dim, out_row, out_head, true));
    if (pos_row < 0 || pos_row > MAX_STRIDE) return fail(SUBMCONV_E_INVALID_ARG, "pos_row = %lld", (long long)pos_row);
    if (n == 0) return SUBMCONV_OK;
    if (!x || !out || !positions || (pairs && !freqs)) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype);
    if (!aligned_to(x, es) || !aligned_to(out, es) || !aligned_to(positions, 4) || !aligned_to(freqs, 4))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const bool same = x == out && (n == 1 || x_row == out_row) && (heads == 1 || x_head == out_head);  // in place
    const Range r[] = {range3("x", same ? nullptr : x, n, heads, dim, x_row, x_head, es, false),
                       range3("out", out, n, heads, dim, out_row, out_head, es, true),
                       range2("positions", positions, n, axes, pos_row, 4, false),
                       range1("freqs", freqs, (size_t)pairs * 4, false)};
    SC_CHECK(ranges_check(r, 4));
    return rotary(x, x_row, x_head, positions, pos_row, freqs, sections, axes, n, heads, dim, dtype, split, inverse,
                  out, out_row, out_head, (hipStream_t)stream);
}

// Sizes of an attention call, checked, into A (pointers stay zero).  Takes the flag out of dtype.
static int attn_sizes(AttnArgs *A, int32_t entries, int64_t nq, int64_t nk, int32_t heads, int32_t kv_heads,
                      int32_t dim, int32_t &dtype)
{
    *A = AttnArgs{};
    A->out_f32 = dtype >= 0 && (dtype & SUBMCONV_OUT_F32);
    if (A->out_f32) dtype &= ~SUBMCONV_OUT_F32;
    if (!known_dtype(dtype)) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (entries < 1 || entries > 1 << 20) return fail(SUBMCONV_E_INVALID_ARG, "entries = %d outside 1..2^20", entries);
    if (kv_heads < 1 || heads < kv_heads || heads > 1024 || heads % kv_heads)
        return fail(SUBMCONV_E_UNSUPPORTED, "heads = %d, kv_heads = %d: heads must be a multiple of kv_heads, up to 1024", heads, kv_heads);
    if (dim < 8 || dim > SUBMCONV_ATTENTION_MAX_DIM || dim % 8)
        return fail(SUBMCONV_E_UNSUPPORTED, "dim = %d is not a multiple of 8 in 8..%d", dim, SUBMCONV_ATTENTION_MAX_DIM);
    if (nq < 0 || nk < 0 || nq >= MAX_ROWS / heads || nk >= MAX_ROWS / kv_heads)
        return fail(SUBMCONV_E_INVALID_ARG, "nq = %lld, nk = %lld: rows times heads must stay below 2^31", (long long)nq, (long long)nk);
    // a launch holds 2^32 threads: 2^24 blocks, some left for cut tiles
    const int64_t rows = nq * heads > nk * kv_heads ? nq * heads : nk * kv_heads;
    if (rows / 128 + ((int64_t)entries + 2) * kv_heads > (1 << 24) - (1 << 16))
        return fail(SUBMCONV_E_UNSUPPORTED, "%lld tiles and %d entries of %d key heads are more than one launch holds",
                    (long long)(rows / 128), entries, kv_heads);
    A->entries = entries;
    A->nq = nq;
    A->nk = nk;
    A->heads = heads;
    A->kv_heads = kv_heads;
    A->group = heads / kv_heads;
    A->dim = dim;
    return SUBMCONV_OK;
}

size_t submconv_attention_workspace(int32_t entries, int64_t nq, int64_t nk, int32_t heads, int32_t kv_heads,
                                    int32_t dim, int32_t dtype)
{
    AttnArgs A;
    return attn_sizes(&A, entries, nq, nk, heads, kv_heads, dim, dtype) == SUBMCONV_OK ? attention_workspace(A, dtype) : 0;
}

size_t submconv_attention_backward_workspace(int32_t entries, int64_t nq, int64_t nk, int32_t heads, int32_t kv_heads,
                                             int32_t dim, int32_t dtype)
{
    AttnArgs A;
    return attn_sizes(&A, entries, nq, nk, heads, kv_heads, dim, dtype) == SUBMCONV_OK ? attention_backward_workspace(A, dtype) : 0;
}

// Weights are powers of two, so scale log2(e) has to stay finite too.
static int attn_scale_check(float scale)
{
    if (!(scale > 0.0f) || scale > SUBMCONV_ATTENTION_MAX_SCALE)
        return fail(SUBMCONV_E_INVALID_ARG, "scale = %g outside (0, %g]", (double)scale, (double)SUBMCONV_ATTENTION_MAX_SCALE);
    return SUBMCONV_OK;
}

// One [n, heads, dim] tensor of a call: its pointer, distances and range.
static int attn_tensor(const char *what, const void *p, const int64_t *st, int64_t n, int64_t heads, int64_t dim,
                       size_t es, bool written, Heads *h, Range *r)
{
    if (n && !p) return fail(SUBMCONV_E_INVALID_ARG, "%s is NULL", what);
    if (st[0] > SUBMCONV_ATTENTION_MAX_ROW)
        return fail(SUBMCONV_E_UNSUPPORTED, "%s: rows are %lld elements apart, more than 2^22", what, (long long)st[0]);
    if (!aligned_to(p, es)) return fail(SUBMCONV_E_INVALID_ARG, "%s is misaligned", what);
    SC_CHECK(heads_check(what, n, heads, dim, st[0], st[1], written));
    *h = Heads{p, st[0], st[1]};
    *r = range3(what, p, n, heads, dim, st[0], st[1], es, written);
    return SUBMCONV_OK;
}

int submconv_attention(const void *q, const void *k, const void *v, const int64_t *strides, const int32_t *q_offsets,
                       const int32_t *k_offsets, int32_t entries, int64_t nq, int64_t nk, int32_t heads,
                       int32_t kv_heads, int32_t dim, int32_t dtype, float scale, void *out, float *lse,
                       void *workspace, size_t workspace_bytes, void *stream)
{
    AttnArgs A;
    SC_CHECK(attn_sizes(&A, entries, nq, nk, heads, kv_heads, dim, dtype));
    SC_CHECK(attn_scale_check(scale));
    if (!strides) return fail(SUBMCONV_E_INVALID_ARG, "strides is NULL");
    if (nq == 0) return SUBMCONV_OK;
    if (!q_offsets || !k_offsets) return fail(SUBMCONV_E_INVALID_ARG, "offsets are NULL");
    if (!aligned_to(q_offsets, 4) || !aligned_to(k_offsets, 4) || !aligned_to(lse, 4) || !aligned16(workspace))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const size_t es = elem_size(dtype), need = attention_workspace(A, dtype), ob = ((size_t)entries + 1) * 4;
    if (need && (!workspace || workspace_bytes < need))
        return fail(SUBMCONV_E_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    Range r[8];
    SC_CHECK(attn_tensor("q", q, strides, nq, heads, dim, es, false, &A.q, &r[0]));
    SC_CHECK(attn_tensor("k", k, strides + 2, nk, kv_heads, dim, es, false, &A.k, &r[1]));
    SC_CHECK(attn_tensor("v", v, strides + 4, nk, kv_heads, dim, es, false, &A.v, &r[2]));
    SC_CHECK(attn_tensor("out", out, strides + 6, nq, heads, dim, A.out_f32 ? 4 : es, true, &A.out, &r[3]));
    r[4] = range1("lse", lse, (size_t)nq * heads * 4, true);
    r[5] = range1("workspace", workspace, need, true);
    r[6] = range1("q_offsets", q_offsets, ob, false);
    r[7] = range1("k_offsets", k_offsets, ob, false);
    SC_CHECK(ranges_check(r, 8));
    A.q_off = q_offsets;
    A.k_off = k_offsets;
    A.scale = scale;
    A.lse = lse;
    return attention(A, dtype, workspace, (hipStream_t)stream);
}

int submconv_attention_backward(const void *grad, const void *q, const void *k, const void *v, const void *out,
                                const float *lse, const int64_t *strides, const int32_t *q_offsets,
                                const int32_t *k_offsets, int32_t entries, int64_t nq, int64_t nk, int32_t heads,
                                int32_t kv_heads, int32_t dim, int32_t dtype, float scale, void *dq, void *dk,
                                void *dv, void *workspace, size_t workspace_bytes, void *stream)
{
    AttnArgs A;
    SC_CHECK(attn_sizes(&A, entries, nq, nk, heads, kv_heads, dim, dtype));
    SC_CHECK(attn_scale_check(scale));
    if (!strides) return fail(SUBMCONV_E_INVALID_ARG, "strides is NULL");
    if (nq == 0 && nk == 0) return SUBMCONV_OK;
    if (!q_offsets || !k_offsets || (nq && !lse)) return fail(SUBMCONV_E_INVALID_ARG, "offsets or lse are NULL");
    if (!aligned_to(q_offsets, 4) || !aligned_to(k_offsets, 4) || !aligned_to(lse, 4) || !aligned16(workspace))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const size_t es = elem_size(dtype), need = attention_backward_workspace(A, dtype), ob = ((size_t)entries + 1) * 4;
    if (need && (!workspace || workspace_bytes < need))
        return fail(SUBMCONV_E_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    Range r[12];
    SC_CHECK(attn_tensor("grad", grad, strides, nq, heads, dim, es, false, &A.grad, &r[0]));
    SC_CHECK(attn_tensor("q", q, strides + 2, nq, heads, dim, es, false, &A.q, &r[1]));
    SC_CHECK(attn_tensor("k", k, strides + 4, nk, kv_heads, dim, es, false, &A.k, &r[2]));
    SC_CHECK(attn_tensor("v", v, strides + 6, nk, kv_heads, dim, es, false, &A.v, &r[3]));
    SC_CHECK(attn_tensor("out", out, strides + 8, nq, heads, dim, A.out_f32 ? 4 : es, false, &A.out, &r[4]));
    SC_CHECK(attn_tensor("dq", dq, strides + 10, nq, heads, dim, es, true, &A.dq, &r[5]));
    SC_CHECK(attn_tensor("dk", dk, strides + 12, nk, kv_heads, dim, es, true, &A.dk, &r[6]));
    SC_CHECK(attn_tensor("dv", dv, strides + 14, nk, kv_heads, dim, es, true, &A.dv, &r[7]));
    r[8] = range1("lse", lse, (size_t)nq * heads * 4, false);
    r[9] = range1("workspace", workspace, need, true);
    r[10] = range1("q_offsets", q_offsets, ob, false);
    r[11] = range1("k_offsets", k_offsets, ob, false);
    SC_CHECK(ranges_check(r, 12));
    A.q_off = q_offsets;
    A.k_off = k_offsets;
    A.scale = scale;
    A.lse = const_cast<float *>(lse);
    return attention_backward(A, dtype, workspace, (hipStream_t)stream);
}

// Sizes, sections and positions of a call of the heads' norm (axes = 0: no rotation); *pairs is what turns.
static int head_norm_check(int64_t n, int32_t heads, int32_t dim, int32_t dtype, int32_t param_dtype, const void *weight,
                           int32_t weight_rows, int32_t q_heads, const int32_t *sections, int32_t axes, int32_t split,
                           int64_t pos_row, int64_t *pairs)
{
    if (n < 0 || n >= MAX_ROWS) return fail(SUBMCONV_E_INVALID_ARG, "n = %lld outside [0, 2^31)", (long long)n);
    if (!known_dtype(dtype) || !known_dtype(param_dtype)) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d, param_dtype %d", dtype, param_dtype);
    if (dim < 2 || dim > 512 || dim % 2) return fail(SUBMCONV_E_UNSUPPORTED, "dim = %d is not an even number in 2..512", dim);
    if (heads < 1 || heads > 1024) return fail(SUBMCONV_E_UNSUPPORTED, "heads = %d outside 1..1024", heads);
    if (axes < 0 || axes > SUBMCONV_ROTARY_MAX_AXES)
        return fail(SUBMCONV_E_UNSUPPORTED, "axes = %d outside 0..%d", axes, SUBMCONV_ROTARY_MAX_AXES);
    if (split & ~1) return fail(SUBMCONV_E_INVALID_ARG, "split must be 0 or 1");
    if (q_heads < 0 || q_heads > heads) return fail(SUBMCONV_E_INVALID_ARG, "q_heads = %d outside 0..%d", q_heads, heads);
    if (q_heads ? weight_rows != 2 : (weight_rows != 1 && weight_rows != heads))
        return fail(SUBMCONV_E_INVALID_ARG, "weight_rows = %d for %d heads, q_heads = %d", weight_rows, heads, q_heads);
    if (!weight && (weight_rows != 1 || q_heads)) return fail(SUBMCONV_E_INVALID_ARG, "weight is NULL, weight_rows = %d, q_heads = %d", weight_rows, q_heads);
    *pairs = 0;
    if (axes && !sections) return fail(SUBMCONV_E_INVALID_ARG, "sections is NULL");
    for (int a = 0; a < axes; ++a) {
        if (sections[a] < 0) return fail(SUBMCONV_E_INVALID_ARG, "sections[%d] = %d", a, sections[a]);
        *pairs += sections[a];
    }
    if (*pairs > dim / 2) return fail(SUBMCONV_E_INVALID_ARG, "sections hold %lld pairs, a head has %d", (long long)*pairs, dim / 2);
    if (pos_row < 0 || pos_row > MAX_STRIDE) return fail(SUBMCONV_E_INVALID_ARG, "pos_row = %lld", (long long)pos_row);
    return SUBMCONV_OK;
}

static HeadNormArgs head_norm_args(int64_t n, int32_t heads, int32_t dim, const void *weight, int32_t weight_rows, int32_t q_heads,
                                   int32_t param_dtype, const int32_t *positions, int64_t pos_row, const float *freqs,
                                   const int32_t *sections, int32_t axes)
{
    HeadNormArgs A = {};
    A.n = n;
    A.heads = heads;
    A.dim = dim;
    A.w = weight;
    A.weight_rows = weight_rows;
    A.q_heads = q_heads;
    A.pdtype = param_dtype;
    A.pos = positions;
    A.pos_row = pos_row;
    A.freqs = freqs;
    A.ax = rotary_axes(sections, axes);
    return A;
}

int submconv_head_norm_rotary(const void *x, int64_t x_row, int64_t x_head, const void *weight, int32_t weight_rows,
                              int32_t q_heads, int32_t param_dtype, float eps, const int32_t *positions,
                              int64_t pos_row, const float *freqs, const int32_t *sections, int32_t axes, int64_t n,
                              int32_t heads, int32_t dim, int32_t dtype, int32_t split, void *out, int64_t out_row,
                              int64_t out_head, float *rstd, void *stream)
{
    int64_t pairs;
    SC_CHECK(head_norm_check(n, heads, dim, dtype, param_dtype, weight, weight_rows, q_heads, sections, axes, split, pos_row, &pairs));
    if (!(eps >= 0.0f)) return fail(SUBMCONV_E_INVALID_ARG, "eps = %g", (double)eps);
    SC_CHECK(heads_check("x", n, heads, dim, x_row, x_head, false));
    SC_CHECK(heads_check("out", n, heads, dim, out_row, out_head, true));
    if (n == 0) return SUBMCONV_OK;
    if (!x || !out || (pairs && (!positions || !freqs))) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
    if (!aligned_to(x, es) || !aligned_to(out, es) || !aligned_to(weight, ps) || !aligned_to(positions, 4) || !aligned_to(freqs, 4) ||
        !aligned_to(rstd, 4))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const bool same = x == out && (n == 1 || x_row == out_row) && (heads == 1 || x_head == out_head);  // in place
    const Range r[] = {range3("x", same ? nullptr : x, n, heads, dim, x_row, x_head, es, false),
                       range3("out", out, n, heads, dim, out_row, out_head, es, true),
                       range2("positions", pairs ? positions : nullptr, n, axes, pos_row, 4, false),
                       range1("freqs", freqs, (size_t)pairs * 4, false),
                       range1("weight", weight, (size_t)weight_rows * dim * ps, false),
                       range1("rstd", rstd, (size_t)n * heads * 4, true)};
    SC_CHECK(ranges_check(r, 6));
    HeadNormArgs A = head_norm_args(n, heads, dim, weight, weight_rows, q_heads, param_dtype, positions, pos_row, freqs, sections, axes);
    A.x = x;
    A.x_row = x_row;
    A.x_head = x_head;
    A.out = out;
    A.out_row = out_row;
    A.out_head = out_head;
    A.rstd = rstd;
    A.eps = eps;
    return head_norm(A, dtype, split, (hipStream_t)stream);
}

size_t submconv_head_norm_rotary_backward_workspace(int64_t n, int32_t heads, int32_t dim, int32_t dtype,
                                                    int32_t weight_rows, int32_t q_heads)
{
    int64_t pairs;
    const int some = 0;
    if (head_norm_check(n, heads, dim, dtype, SUBMCONV_F32, &some, weight_rows, q_heads, nullptr, 0, 0, 0, &pairs) != SUBMCONV_OK) return 0;
    return head_norm_bwd_workspace(n, heads, dim, dtype, weight_rows, q_heads);
}

int submconv_head_norm_rotary_backward(const void *grad, const void *x, const float *rstd, const void *weight,
                                       int32_t weight_rows, int32_t q_heads, int32_t param_dtype,
                                       const int32_t *positions, int64_t pos_row, const float *freqs,
                                       const int32_t *sections, int32_t axes, const int64_t *strides, int64_t n,
                                       int32_t heads, int32_t dim, int32_t dtype, int32_t split, void *dx,
                                       void *dweight, void *workspace, size_t workspace_bytes, void *stream)
{
    int64_t pairs;
    SC_CHECK(head_norm_check(n, heads, dim, dtype, param_dtype, weight, weight_rows, q_heads, sections, axes, split, pos_row, &pairs));
    if (!strides) return fail(SUBMCONV_E_INVALID_ARG, "strides is NULL");
    SC_CHECK(heads_check("grad", n, heads, dim, strides[0], strides[1], false));
    SC_CHECK(heads_check("x", n, heads, dim, strides[2], strides[3], false));
    SC_CHECK(heads_check("dx", n, heads, dim, strides[4], strides[5], true));
    if (n && (!grad || !x || !rstd || !dx || (pairs && (!positions || !freqs)))) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype), ps = elem_size(param_dtype), wb = (size_t)weight_rows * dim * ps;
    if (!aligned_to(grad, es) || !aligned_to(x, es) || !aligned_to(dx, es) || !aligned_to(weight, ps) || !aligned_to(dweight, ps) ||
        !aligned_to(positions, 4) || !aligned_to(freqs, 4) || !aligned_to(rstd, 4) || !aligned16(workspace))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const size_t need = dweight ? head_norm_bwd_workspace(n, heads, dim, dtype, weight_rows, q_heads) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return fail(SUBMCONV_E_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    const bool same = grad == dx && (n <= 1 || strides[0] == strides[4]) && (heads == 1 || strides[1] == strides[5]);  // in place
    const Range r[] = {range3("grad", same ? nullptr : grad, n, heads, dim, strides[0], strides[1], es, false),
                       range3("x", x, n, heads, dim, strides[2], strides[3], es, false),
                       range3("dx", dx, n, heads, dim, strides[4], strides[5], es, true),
                       range2("positions", pairs ? positions : nullptr, n, axes, pos_row, 4, false),
                       range1("freqs", freqs, (size_t)pairs * 4, false), range1("weight", weight, wb, false),
                       range1("rstd", rstd, (size_t)n * heads * 4, false), range1("dweight", dweight, wb, true),
                       range1("workspace", workspace, need, true)};
    SC_CHECK(ranges_check(r, 9));
    HeadNormArgs A = head_norm_args(n, heads, dim, weight, weight_rows, q_heads, param_dtype, positions, pos_row, freqs, sections, axes);
    A.g = grad;
    A.g_row = strides[0];
    A.g_head = strides[1];
    A.x = x;
    A.x_row = strides[2];
    A.x_head = strides[3];
    A.out = dx;
    A.out_row = strides[4];
    A.out_head = strides[5];
    A.rstd = const_cast<float *>(rstd);
    A.partial = (float *)workspace;
    return head_norm_backward(A, dtype, split, dweight, (hipStream_t)stream);
}

static int route_check(int64_t n, int32_t experts, int32_t k, int32_t dtype, int32_t normalize, int64_t row)
{
    if (!known_dtype(dtype)) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (experts < 1 || experts > SUBMCONV_ROUTE_MAX_EXPERTS)
        return fail(SUBMCONV_E_UNSUPPORTED, "experts = %d outside 1..%d", experts, SUBMCONV_ROUTE_MAX_EXPERTS);
    if (k < 1 || k > SUBMCONV_ROUTE_MAX_K || k > experts)
        return fail(SUBMCONV_E_UNSUPPORTED, "k = %d outside 1..%d, or more than %d experts", k, SUBMCONV_ROUTE_MAX_K, experts);
    if (n < 0 || n >= MAX_ROWS / k) return fail(SUBMCONV_E_INVALID_ARG, "n = %lld: n k must stay in [0, 2^31)", (long long)n);
    if (normalize & ~1) return fail(SUBMCONV_E_INVALID_ARG, "normalize must be 0 or 1");
    return row_check("logits", row, 0);
}

size_t submconv_route_workspace(int64_t n, int32_t experts, int32_t k)
{
    return route_check(n, experts, k, SUBMCONV_F32, 0, 0) == SUBMCONV_OK ? route_workspace(n, experts, k) : 0;
}

int submconv_route(const void *logits, int64_t row, int64_t n, int32_t experts, int32_t k, int32_t dtype,
                   int32_t normalize, int32_t *chosen, float *gates, int32_t *offsets, int32_t *rows, int32_t *slots,
                   void *workspace, size_t workspace_bytes, void *stream)
{
    SC_CHECK(route_check(n, experts, k, dtype, normalize, row));
    if (!offsets || (n && (!logits || !chosen || !gates || !rows || !slots))) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype), need = route_workspace(n, experts, k), pb = (size_t)n * k * 4;
    if (!aligned_to(logits, es) || !aligned_to(chosen, 4) || !aligned_to(gates, 4) || !aligned_to(offsets, 4) || !aligned_to(rows, 4) ||
        !aligned_to(slots, 4) || !aligned16(workspace))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    if (need && (!workspace || workspace_bytes < need))
        return fail(SUBMCONV_E_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    const Range r[] = {range2("logits", logits, n, experts, row, es, false), range1("chosen", chosen, pb, true),
                       range1("gates", gates, pb, true), range1("offsets", offsets, ((size_t)experts + 1) * 4, true),
                       range1("rows", rows, pb, true), range1("slots", slots, pb, true), range1("workspace", workspace, need, true)};
    SC_CHECK(ranges_check(r, 7));
    if (n == 0) return route_none(offsets, experts, (hipStream_t)stream);
    return route(logits, row, n, experts, k, dtype, normalize, chosen, gates, offsets, rows, slots, workspace, (hipStream_t)stream);
}

int submconv_route_backward(const float *grad, const void *logits, int64_t row, int64_t n, int32_t experts, int32_t k,
                            int32_t dtype, int32_t normalize, const int32_t *chosen, const float *gates, void *dlogits,
                            int64_t out_row, void *stream)
{
    SC_CHECK(route_check(n, experts, k, dtype, normalize, row));
    SC_CHECK(row_check("dlogits", out_row, experts));
    if (n == 0) return SUBMCONV_OK;
    if (!grad || !chosen || !gates || !dlogits || (!normalize && !logits)) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype), pb = (size_t)n * k * 4;
    if (!aligned_to(logits, es) || !aligned_to(dlogits, es) || !aligned_to(chosen, 4) || !aligned_to(gates, 4) || !aligned_to(grad, 4))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const Range r[] = {range2("logits", logits, n, experts, row, es, false), range2("dlogits", dlogits, n, experts, out_row, es, true),
                       range1("grad", grad, pb, false), range1("chosen", chosen, pb, false), range1("gates", gates, pb, false)};
    SC_CHECK(ranges_check(r, 5));
    return route_backward(grad, logits, row, n, experts, k, dtype, normalize, chosen, gates, dlogits, out_row, (hipStream_t)stream);
}

constexpr int64_t MAX_POSITIONS = MAX_ROWS - (1 << 16);  // a tile's row numbers stay below 2^31
constexpr int MAX_WIDTH = 1 << 16, MAX_GROUPS = 1 << 16;

static int linear_check(int32_t groups, int64_t n, int64_t nx, int32_t cin, int32_t cout, int32_t dtype, bool forward, bool dx, bool dw)
{
    if (!known_dtype(dtype)) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (n < 0 || n >= MAX_POSITIONS || nx < 0 || nx >= MAX_POSITIONS)
        return fail(SUBMCONV_E_INVALID_ARG, "n = %lld or nx = %lld outside [0, 2^31 - 2^16)", (long long)n, (long long)nx);
    if (cin < 1 || cin > MAX_WIDTH || cout < 1 || cout > MAX_WIDTH)
        return fail(SUBMCONV_E_UNSUPPORTED, "cin = %d, cout = %d outside 1..%d", cin, cout, MAX_WIDTH);
    if (groups < 1 || groups > MAX_GROUPS) return fail(SUBMCONV_E_INVALID_ARG, "groups = %d outside 1..%d", groups, MAX_GROUPS);
    if ((int64_t)groups * cin * cout >= int64_t(1) << 40) return fail(SUBMCONV_E_UNSUPPORTED, "groups cin cout reaches 2^40");
    for (int kind = LINEAR_Y; kind <= LINEAR_DW; ++kind)
        if ((kind == LINEAR_Y ? forward : (kind == LINEAR_DX ? dx : dw)) && linear_blocks(n, groups, cin, cout, dtype, kind) >= 1 << 24)
            return fail(SUBMCONV_E_UNSUPPORTED, "%lld tiles are more than one launch holds", (long long)linear_blocks(n, groups, cin, cout, dtype, kind));
    return SUBMCONV_OK;
}

int submconv_grouped_linear(const void *x, int64_t x_row, int64_t nx, const int32_t *rows, const void *weight,
                            const float *bias, const int32_t *offsets, int32_t groups, int64_t n, int32_t cin,
                            int32_t cout, int32_t dtype, void *out, int64_t out_row, void *stream)
{
    SC_CHECK(linear_check(groups, n, nx, cin, cout, dtype, true, false, false));
    SC_CHECK(row_check("x", x_row, 0));
    SC_CHECK(row_check("out", out_row, cout));
    if (n == 0) return SUBMCONV_OK;
    if (!rows && nx != n) return fail(SUBMCONV_E_INVALID_ARG, "nx = %lld and n = %lld differ, rows is NULL", (long long)nx, (long long)n);
    if ((nx && !x) || !weight || !offsets || !out) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype), gc = (size_t)groups * cout;
    if (!aligned_to(x, es) || !aligned_to(weight, es) || !aligned_to(out, es) || !aligned_to(rows, 4) || !aligned_to(bias, 4) || !aligned_to(offsets, 4))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const Range r[] = {range2("x", x, nx, cin, x_row, es, false), range2("out", out, n, cout, out_row, es, true),
                       range1("rows", rows, (size_t)n * 4, false), range1("weight", weight, gc * cin * es, false),
                       range1("bias", bias, gc * 4, false), range1("offsets", offsets, ((size_t)groups + 1) * 4, false)};
    SC_CHECK(ranges_check(r, 6));
    LinearArgs A = {};
    A.x = x;
    A.x_row = x_row;
    A.nx = (int32_t)nx;
    A.rows = rows;
    A.w = weight;
    A.bias = bias;
    A.off = offsets;
    A.groups = groups;
    A.n = (int32_t)n;
    A.cin = cin;
    A.cout = cout;
    A.out = out;
    A.out_row = out_row;
    return grouped_linear(A, dtype, LINEAR_Y, nullptr, (hipStream_t)stream);
}

size_t submconv_grouped_linear_backward_workspace(int32_t groups, int64_t n, int32_t cin, int32_t cout, int32_t dtype)
{
    if (linear_check(groups, n, n, cin, cout, dtype, false, false, true) != SUBMCONV_OK) return 0;
    return linear_dw_workspace(n, groups, cin, cout, dtype);
}

int submconv_grouped_linear_backward(const void *grad, int64_t grad_row, const void *x, int64_t x_row, int64_t nx,
                                     const int32_t *rows, const void *weight, const int32_t *offsets, int32_t groups,
                                     int64_t n, int32_t cin, int32_t cout, int32_t dtype, void *dx, int64_t dx_row,
                                     void *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                                     void *stream)
{
    SC_CHECK(linear_check(groups, n, nx, cin, cout, dtype, false, dx != nullptr, dweight != nullptr));
    SC_CHECK(row_check("grad", grad_row, 0));
    SC_CHECK(row_check("x", x_row, 0));
    SC_CHECK(row_check("dx", dx_row, cin));
    if (!rows && dweight && n && nx != n) return fail(SUBMCONV_E_INVALID_ARG, "nx = %lld and n = %lld differ, rows is NULL", (long long)nx, (long long)n);
    if (dbias && !dweight) return fail(SUBMCONV_E_INVALID_ARG, "dbias without dweight");
    if (!dx && !dweight) return SUBMCONV_OK;
    if ((n && !grad) || !offsets || (dx && !weight) || (dweight && n && nx && !x)) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype), gc = (size_t)groups * cout;
    if (!aligned_to(grad, es) || !aligned_to(x, es) || !aligned_to(weight, es) || !aligned_to(dx, es) || !aligned_to(dweight, es) ||
        !aligned_to(dbias, 4) || !aligned_to(rows, 4) || !aligned_to(offsets, 4) || !aligned16(workspace))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const size_t need = dweight ? linear_dw_workspace(n, groups, cin, cout, dtype) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return fail(SUBMCONV_E_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    const Range r[] = {range2("grad", grad, n, cout, grad_row, es, false), range2("x", dweight ? x : nullptr, nx, cin, x_row, es, false),
                       range2("dx", dx, n, cin, dx_row, es, true), range1("rows", dweight ? rows : nullptr, (size_t)n * 4, false),
                       range1("weight", dx ? weight : nullptr, gc * cin * es, false), range1("offsets", offsets, ((size_t)groups + 1) * 4, false),
                       range1("dweight", dweight, gc * cin * es, true), range1("dbias", dbias, gc * 4, true),
                       range1("workspace", workspace, need, true)};
    SC_CHECK(ranges_check(r, 9));
    LinearArgs A = {};
    A.g = grad;
    A.g_row = grad_row;
    A.x = x;
    A.x_row = x_row;
    A.nx = (int32_t)nx;
    A.rows = rows;
    A.w = weight;
    A.off = offsets;
    A.groups = groups;
    A.n = (int32_t)n;
    A.cin = cin;
    A.cout = cout;
    if (dx && n) {
        A.out = dx;
        A.out_row = dx_row;
        SC_CHECK(grouped_linear(A, dtype, LINEAR_DX, nullptr, (hipStream_t)stream));
    }
    if (dweight) {
        A.out = dweight;
        A.db = dbias;
        SC_CHECK(grouped_linear(A, dtype, LINEAR_DW, workspace, (hipStream_t)stream));
    }
    return SUBMCONV_OK;
}

static int combine_check(int64_t np, int64_t n, int32_t k, int32_t c, int32_t dtype)
{
    if (!known_dtype(dtype)) return fail(SUBMCONV_E_UNSUPPORTED, "dtype %d", dtype);
    if (k < 1 || k > SUBMCONV_ROUTE_MAX_K) return fail(SUBMCONV_E_UNSUPPORTED, "k = %d outside 1..%d", k, SUBMCONV_ROUTE_MAX_K);
    if (c < 1 || c > MAX_WIDTH) return fail(SUBMCONV_E_UNSUPPORTED, "c = %d outside 1..%d", c, MAX_WIDTH);
    if (n < 0 || n >= MAX_ROWS || np < 0 || np >= MAX_ROWS)
        return fail(SUBMCONV_E_INVALID_ARG, "n = %lld or np = %lld outside [0, 2^31)", (long long)n, (long long)np);
    return SUBMCONV_OK;
}

int submconv_combine(const void *y, int64_t y_row, int64_t np, const int32_t *slots, const float *gates, int64_t n,
                     int32_t k, int32_t c, int32_t dtype, void *out, int64_t out_row, void *stream)
{
    SC_CHECK(combine_check(np, n, k, c, dtype));
    SC_CHECK(row_check("y", y_row, 0));
    SC_CHECK(row_check("out", out_row, c));
    if (n == 0) return SUBMCONV_OK;
    if ((np && !y) || !slots || !out) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype), pb = (size_t)n * k * 4;
    if (!aligned_to(y, es) || !aligned_to(out, es) || !aligned_to(slots, 4) || !aligned_to(gates, 4))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const Range r[] = {range2("y", y, np, c, y_row, es, false), range2("out", out, n, c, out_row, es, true),
                       range1("slots", slots, pb, false), range1("gates", gates, pb, false)};
    SC_CHECK(ranges_check(r, 4));
    return combine(y, y_row, np, slots, gates, n, k, c, dtype, out, out_row, (hipStream_t)stream);
}

int submconv_combine_backward(const void *grad, int64_t grad_row, const void *y, int64_t y_row, int64_t np,
                              const int32_t *slots, const int32_t *rows, const float *gates, int64_t n, int32_t k,
                              int32_t c, int32_t dtype, void *dy, int64_t dy_row, float *dgates, void *stream)
{
    SC_CHECK(combine_check(np, n, k, c, dtype));
    SC_CHECK(row_check("grad", grad_row, 0));
    SC_CHECK(row_check("y", y_row, 0));
    SC_CHECK(row_check("dy", dy_row, c));
    if ((!dy || np == 0) && (!dgates || n == 0)) return SUBMCONV_OK;
    if ((n && (!grad || !slots)) || (dy && np && !rows) || (dgates && np && !y)) return fail(SUBMCONV_E_INVALID_ARG, "NULL tensor pointer");
    const size_t es = elem_size(dtype), pb = (size_t)n * k * 4;
    if (!aligned_to(grad, es) || !aligned_to(y, es) || !aligned_to(dy, es) || !aligned_to(slots, 4) || !aligned_to(rows, 4) ||
        !aligned_to(gates, 4) || !aligned_to(dgates, 4))
        return fail(SUBMCONV_E_INVALID_ARG, "misaligned pointer");
    const Range r[] = {range2("grad", grad, n, c, grad_row, es, false), range2("y", dgates ? y : nullptr, np, c, y_row, es, false),
                       range2("dy", dy, np, c, dy_row, es, true), range1("slots", slots, pb, false),
                       range1("rows", dy ? rows : nullptr, (size_t)np * 4, false), range1("gates", gates, pb, false),
                       range1("dgates", dgates, pb, true)};
    SC_CHECK(ranges_check(r, 7));
    return combine_backward(grad, grad_row, y, y_row, np, slots, rows, gates, n, k, c, dtype, dy, dy_row, dgates, (hipStream_t)stream);
}

int submconv_release_cache(int32_t device)
{
    std::lock_guard<std::mutex> lock(g_cache_mu);
    int cur = 0;
    if (hipGetDevice(&cur) != hipSuccess) return fail(SUBMCONV_E_HIP, "hipGetDevice failed");
    release_cached(device);
    (void)hipSetDevice(cur);
    (void)hipDeviceSynchronize();  // the frees are queued on the null stream; let them land
    return SUBMCONV_OK;
}

int submconv_set_cache_limit(int64_t bytes)
{
    if (bytes < 0) return fail(SUBMCONV_E_INVALID_ARG, "cache limit %lld < 0", (long long)bytes);
    std::lock_guard<std::mutex> lock(g_cache_mu);
    g_cap = (size_t)bytes;
    int cur = 0;
    if (hipGetDevice(&cur) != hipSuccess) return fail(SUBMCONV_E_HIP, "hipGetDevice failed");
    for (int d = 0; d < 64; ++d)  // shrink: drop cached blocks of devices above the new limit
        if (g_cached[d] > g_cap) release_cached(d);
    (void)hipSetDevice(cur);
    return SUBMCONV_OK;
}

}  // extern "C"
