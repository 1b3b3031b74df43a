// api.cu -- the C ABI of libgdn (declared in include/gdn.h): host-side validation, choice of kernel
// configuration, launch, and error reporting.  No device memory is allocated here.
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "gdn.h"
#include "launch.h"

namespace {

thread_local char g_last_error[512] = "";

gdn_status fail(gdn_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return s;
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Two byte ranges overlap without being identical.
bool partial_overlap(const void* a, size_t na, const void* b, size_t nb) {
    const char* pa = static_cast<const char*>(a);
    const char* pb = static_cast<const char*>(b);
    if (pa == pb) return false;
    return pa < pb + nb && pb < pa + na;
}

bool any_overlap(const void* a, size_t na, const void* b, size_t nb) {
    const char* pa = static_cast<const char*>(a);
    const char* pb = static_cast<const char*>(b);
    return na > 0 && nb > 0 && pa < pb + nb && pb < pa + na;
}

gdn_status launched(const char* what) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
    g_last_error[0] = '\0';
    return GDN_OK;
}

#define REQUIRE(cond, status, ...)                    \
    do {                                              \
        if (!(cond)) return fail(status, __VA_ARGS__); \
    } while (0)

}  // namespace

extern "C" {

const char* gdn_status_string(gdn_status s) {
    switch (s) {
        case GDN_OK: return "ok";
        case GDN_ERR_INVALID_ARG: return "invalid argument";
        case GDN_ERR_UNSUPPORTED: return "unsupported shape or option";
        case GDN_ERR_CUDA: return "CUDA error";
        case GDN_ERR_TIMEOUT: return "device wait timed out";
    }
    return "unknown status";
}

const char* gdn_last_error(void) { return g_last_error; }

// ------------------------------------------------------------------------------------------------
gdn_status gdn_decode_step(const float* state_in, float* state_out, const void* q, const void* k,
                           const void* v, const float* g, const void* beta, void* y,
                           gdn_dtype y_dtype, int B, int Hk, int Hv, int Dk, int Dv, float scale,
                           gdn_stream_t stream) {
    REQUIRE(B >= 0 && Hk >= 1 && Hv >= 1 && Dk >= 1 && Dv >= 1, GDN_ERR_INVALID_ARG,
            "gdn_decode_step: sizes must be B >= 0 and Hk, Hv, Dk, Dv >= 1 (got B=%d Hk=%d Hv=%d "
            "Dk=%d Dv=%d)", B, Hk, Hv, Dk, Dv);
    REQUIRE(Hv % Hk == 0, GDN_ERR_INVALID_ARG, "gdn_decode_step: Hv (%d) must be a multiple of Hk (%d)",
            Hv, Hk);
    REQUIRE(y_dtype == GDN_BF16 || y_dtype == GDN_F32, GDN_ERR_INVALID_ARG,
            "gdn_decode_step: y_dtype must be GDN_BF16 or GDN_F32");
    REQUIRE(Dk == 64 || Dk == 128 || Dk == 256, GDN_ERR_UNSUPPORTED,
            "gdn_decode_step: Dk must be 64, 128 or 256 (got %d)", Dk);
    if (B == 0) return GDN_OK;
    REQUIRE(state_in && state_out && q && k && v && g && beta && y, GDN_ERR_INVALID_ARG,
            "gdn_decode_step: null pointer");
    const size_t sbytes = size_t(B) * Hv * Dv * Dk * sizeof(float);
    REQUIRE(!partial_overlap(state_in, sbytes, state_out, sbytes), GDN_ERR_INVALID_ARG,
            "gdn_decode_step: state_out partially overlaps state_in");
    REQUIRE(aligned(state_in, 16) && aligned(state_out, 16), GDN_ERR_INVALID_ARG,
            "gdn_decode_step: state buffers must be 16-byte aligned");
    REQUIRE(aligned(q, 8) && aligned(k, 8), GDN_ERR_INVALID_ARG,
            "gdn_decode_step: q and k must be 8-byte aligned");
    REQUIRE(aligned(y, y_dtype == GDN_F32 ? 4 : 2) && aligned(v, 2) && aligned(beta, 2) && aligned(g, 4),
            GDN_ERR_INVALID_ARG, "gdn_decode_step: misaligned v, beta, g or y");
    const size_t yb = size_t(B) * Hv * Dv * (y_dtype == GDN_F32 ? 4 : 2);
    REQUIRE(!any_overlap(y, yb, state_out, sbytes), GDN_ERR_INVALID_ARG,
            "gdn_decode_step: y overlaps state_out");
    const long long heads = (long long)B * Hv;
    REQUIRE(heads * ((Dv + 31) / 32) < (1LL << 31), GDN_ERR_UNSUPPORTED, "gdn_decode_step: grid too large");

    gdn::DecodeArgs a;
    a.state_in = state_in;
    a.state_out = state_out;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.g = g;
    a.beta = static_cast<const uint16_t*>(beta);
    a.y = y;
    a.y_f32 = y_dtype == GDN_F32;
    a.Hk = Hk;
    a.Hv = Hv;
    a.Dv = Dv;
    a.scale = scale;
    a.tiles = 0;
    a.slots = nullptr;
    a.pool_size = 0;
    a.status = nullptr;
    gdn::launch_decode(a, B, Dk, static_cast<cudaStream_t>(stream));
    return launched("gdn_decode_step");
}

// ------------------------------------------------------------------------------------------------
gdn_status gdn_decode_multi(const float* state_in, float* state_out, const void* q, const void* k,
                            const void* v, const float* g, const void* beta, void* y,
                            gdn_dtype y_dtype, int B, int T, int Hk, int Hv, int Dk, int Dv,
                            float scale, gdn_stream_t stream) {
    REQUIRE(B >= 0 && T >= 0 && Hk >= 1 && Hv >= 1 && Dk >= 1 && Dv >= 1, GDN_ERR_INVALID_ARG,
            "gdn_decode_multi: sizes must be B, T >= 0 and Hk, Hv, Dk, Dv >= 1");
    REQUIRE(Hv % Hk == 0, GDN_ERR_INVALID_ARG, "gdn_decode_multi: Hv (%d) must be a multiple of Hk (%d)",
            Hv, Hk);
    REQUIRE(y_dtype == GDN_BF16 || y_dtype == GDN_F32, GDN_ERR_INVALID_ARG,
            "gdn_decode_multi: y_dtype must be GDN_BF16 or GDN_F32");
    REQUIRE(Dk == 64 || Dk == 128 || Dk == 256, GDN_ERR_UNSUPPORTED,
            "gdn_decode_multi: Dk must be 64, 128 or 256 (got %d)", Dk);
    if (B == 0 || T == 0) return GDN_OK;
    REQUIRE(state_in && state_out && q && k && v && g && beta && y, GDN_ERR_INVALID_ARG,
            "gdn_decode_multi: null pointer");
    const size_t sbytes = size_t(B) * Hv * Dv * Dk * sizeof(float);
    REQUIRE(!partial_overlap(state_in, sbytes, state_out, sbytes), GDN_ERR_INVALID_ARG,
            "gdn_decode_multi: state_out partially overlaps state_in");
    REQUIRE(aligned(state_in, 16) && aligned(state_out, 16) && aligned(q, 8) && aligned(k, 8),
            GDN_ERR_INVALID_ARG, "gdn_decode_multi: state must be 16-byte, q and k 8-byte aligned");
    REQUIRE(aligned(y, y_dtype == GDN_F32 ? 4 : 2) && aligned(v, 2) && aligned(beta, 2) && aligned(g, 4),
            GDN_ERR_INVALID_ARG, "gdn_decode_multi: misaligned v, beta, g or y");
    const size_t yb = size_t(B) * T * Hv * Dv * (y_dtype == GDN_F32 ? 4 : 2);
    REQUIRE(!any_overlap(y, yb, state_out, sbytes), GDN_ERR_INVALID_ARG, "gdn_decode_multi: y overlaps state_out");
    REQUIRE((long long)B * Hv * ((Dv + 31) / 32) < (1LL << 31), GDN_ERR_UNSUPPORTED,
            "gdn_decode_multi: grid too large");
    gdn::DecodeMultiArgs a;
    a.state_in = state_in;
    a.state_out = state_out;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.g = g;
    a.beta = static_cast<const uint16_t*>(beta);
    a.y = y;
    a.y_f32 = y_dtype == GDN_F32;
    a.T = T;
    a.Hk = Hk;
    a.Hv = Hv;
    a.Dv = Dv;
    a.tiles = 0;
    a.scale = scale;
    gdn::launch_decode_multi(a, B, Dk, static_cast<cudaStream_t>(stream));
    return launched("gdn_decode_multi");
}

// ------------------------------------------------------------------------------------------------
gdn_status gdn_decode_step_pooled(float* state_pool, int pool_size, const int64_t* cache_indices,
                                  const void* q, const void* k, const void* v, const float* g,
                                  const void* beta, void* y, gdn_dtype y_dtype, int B, int Hk, int Hv,
                                  int Dk, int Dv, float scale, int32_t* dev_status,
                                  gdn_stream_t stream) {
    REQUIRE(B >= 0 && pool_size >= 0 && Hk >= 1 && Hv >= 1 && Dk >= 1 && Dv >= 1, GDN_ERR_INVALID_ARG,
            "gdn_decode_step_pooled: sizes must be B, pool_size >= 0 and Hk, Hv, Dk, Dv >= 1");
    REQUIRE(Hv % Hk == 0, GDN_ERR_INVALID_ARG,
            "gdn_decode_step_pooled: Hv (%d) must be a multiple of Hk (%d)", Hv, Hk);
    REQUIRE(y_dtype == GDN_BF16 || y_dtype == GDN_F32, GDN_ERR_INVALID_ARG,
            "gdn_decode_step_pooled: y_dtype must be GDN_BF16 or GDN_F32");
    REQUIRE(Dk == 64 || Dk == 128 || Dk == 256, GDN_ERR_UNSUPPORTED,
            "gdn_decode_step_pooled: Dk must be 64, 128 or 256 (got %d)", Dk);
    if (B == 0) return GDN_OK;
    REQUIRE(state_pool && cache_indices && q && k && v && g && beta && y && dev_status,
            GDN_ERR_INVALID_ARG, "gdn_decode_step_pooled: null pointer");
    REQUIRE(aligned(state_pool, 16) && aligned(q, 8) && aligned(k, 8) && aligned(cache_indices, 8) &&
                aligned(dev_status, 4),
            GDN_ERR_INVALID_ARG, "gdn_decode_step_pooled: misaligned argument");
    REQUIRE(aligned(y, y_dtype == GDN_F32 ? 4 : 2) && aligned(v, 2) && aligned(beta, 2) && aligned(g, 4),
            GDN_ERR_INVALID_ARG, "gdn_decode_step_pooled: misaligned v, beta, g or y");
    const size_t pbytes = size_t(pool_size) * Hv * Dv * Dk * sizeof(float);
    const size_t yb = size_t(B) * Hv * Dv * (y_dtype == GDN_F32 ? 4 : 2);
    REQUIRE(!any_overlap(y, yb, state_pool, pbytes), GDN_ERR_INVALID_ARG,
            "gdn_decode_step_pooled: y overlaps state_pool");
    REQUIRE((long long)B * Hv * ((Dv + 31) / 32) < (1LL << 31), GDN_ERR_UNSUPPORTED,
            "gdn_decode_step_pooled: grid too large");
    gdn::DecodeArgs a;
    a.state_in = state_pool;
    a.state_out = state_pool;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.g = g;
    a.beta = static_cast<const uint16_t*>(beta);
    a.y = y;
    a.y_f32 = y_dtype == GDN_F32;
    a.Hk = Hk;
    a.Hv = Hv;
    a.Dv = Dv;
    a.scale = scale;
    a.tiles = 0;
    a.slots = cache_indices;
    a.pool_size = pool_size;
    a.status = dev_status;
    gdn::launch_decode(a, B, Dk, static_cast<cudaStream_t>(stream));
    return launched("gdn_decode_step_pooled");
}

// ------------------------------------------------------------------------------------------------
gdn_status comba_decode_step(const float* state, float* state_new, const void* q, const void* k,
                             const void* v, const void* p, const void* beta, const float* g,
                             void* o, gdn_dtype o_dtype, int B, int H, int K, int V, float scale,
                             gdn_stream_t stream) {
    REQUIRE(B >= 0 && H >= 1 && K >= 1 && V >= 1, GDN_ERR_INVALID_ARG,
            "comba_decode_step: sizes must be B >= 0 and H, K, V >= 1 (got B=%d H=%d K=%d V=%d)", B, H,
            K, V);
    REQUIRE(o_dtype == GDN_BF16 || o_dtype == GDN_F32, GDN_ERR_INVALID_ARG,
            "comba_decode_step: o_dtype must be GDN_BF16 or GDN_F32");
    REQUIRE((K == 64 || K == 128) && (V == 64 || V == 128), GDN_ERR_UNSUPPORTED,
            "comba_decode_step: K and V must each be 64 or 128 (got K=%d V=%d)", K, V);
    if (B == 0) return GDN_OK;
    REQUIRE(state && state_new && q && k && v && p && beta && g && o, GDN_ERR_INVALID_ARG,
            "comba_decode_step: null pointer");
    const size_t sbytes = size_t(B) * H * K * V * sizeof(float);
    REQUIRE(!partial_overlap(state, sbytes, state_new, sbytes), GDN_ERR_INVALID_ARG,
            "comba_decode_step: state_new partially overlaps state");
    REQUIRE(aligned(state, 16) && aligned(state_new, 16), GDN_ERR_INVALID_ARG,
            "comba_decode_step: state buffers must be 16-byte aligned");
    REQUIRE(aligned(q, 8) && aligned(k, 8) && aligned(p, 8) && aligned(v, 8), GDN_ERR_INVALID_ARG,
            "comba_decode_step: q, k, p and v must be 8-byte aligned");
    REQUIRE(aligned(o, o_dtype == GDN_F32 ? 16 : 8) && aligned(beta, 2) && aligned(g, 4),
            GDN_ERR_INVALID_ARG, "comba_decode_step: misaligned o, beta or g");
    const size_t ob = size_t(B) * H * V * (o_dtype == GDN_F32 ? 4 : 2);
    REQUIRE(!any_overlap(o, ob, state_new, sbytes), GDN_ERR_INVALID_ARG,
            "comba_decode_step: o overlaps state_new");
    REQUIRE((long long)B * H < (1LL << 31), GDN_ERR_UNSUPPORTED, "comba_decode_step: grid too large");

    gdn::CombaArgs a;
    a.state = state;
    a.state_new = state_new;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.p = static_cast<const uint16_t*>(p);
    a.beta = static_cast<const uint16_t*>(beta);
    a.g = g;
    a.o = o;
    a.o_f32 = o_dtype == GDN_F32;
    a.scale = scale;
    gdn::launch_comba(a, B * H, K, V, static_cast<cudaStream_t>(stream));
    return launched("comba_decode_step");
}

gdn_status comba_forward(float* state, const void* q, const void* k, const void* v, const void* p,
                         const void* beta, const float* g, void* o, gdn_dtype o_dtype, int B, int T, int H,
                         int K, int V, float scale, gdn_stream_t stream) {
    REQUIRE(B >= 0 && T >= 0 && H >= 1 && K >= 1 && V >= 1, GDN_ERR_INVALID_ARG,
            "comba_forward: sizes must be B, T >= 0 and H, K, V >= 1 (got B=%d T=%d H=%d K=%d V=%d)", B, T, H,
            K, V);
    REQUIRE(o_dtype == GDN_BF16 || o_dtype == GDN_F32, GDN_ERR_INVALID_ARG,
            "comba_forward: o_dtype must be GDN_BF16 or GDN_F32");
    REQUIRE((K == 64 || K == 128) && (V == 64 || V == 128), GDN_ERR_UNSUPPORTED,
            "comba_forward: K and V must each be 64 or 128 (got K=%d V=%d)", K, V);
    if (B == 0) return GDN_OK;
    REQUIRE(state, GDN_ERR_INVALID_ARG, "comba_forward: null state");
    REQUIRE(T == 0 || (q && k && v && p && beta && g && o), GDN_ERR_INVALID_ARG, "comba_forward: null pointer");
    REQUIRE(aligned(state, 16), GDN_ERR_INVALID_ARG, "comba_forward: state must be 16-byte aligned");
    REQUIRE(aligned(q, 8) && aligned(k, 8) && aligned(p, 8) && aligned(v, 8), GDN_ERR_INVALID_ARG,
            "comba_forward: q, k, p and v must be 8-byte aligned");
    REQUIRE(aligned(o, o_dtype == GDN_F32 ? 16 : 8) && aligned(beta, 2) && aligned(g, 4), GDN_ERR_INVALID_ARG,
            "comba_forward: misaligned o, beta or g");
    const size_t sbytes = size_t(B) * H * K * V * sizeof(float);
    const size_t ob = size_t(B) * T * H * V * (o_dtype == GDN_F32 ? 4 : 2);
    REQUIRE(!any_overlap(o, ob, state, sbytes), GDN_ERR_INVALID_ARG, "comba_forward: o overlaps state");
    REQUIRE((long long)B * H < (1LL << 31) && (long long)B * T * H * (K > V ? K : V) < (1LL << 62),
            GDN_ERR_UNSUPPORTED, "comba_forward: sizes too large");

    gdn::CombaFwdArgs a;
    a.state = state;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.p = static_cast<const uint16_t*>(p);
    a.beta = static_cast<const uint16_t*>(beta);
    a.g = g;
    a.o = o;
    a.o_f32 = o_dtype == GDN_F32;
    a.T = T;
    a.H = H;
    a.scale = scale;
    gdn::launch_comba_forward(a, B * H, K, V, static_cast<cudaStream_t>(stream));
    return launched("comba_forward");
}

}  // extern "C"

// ------------------------------------------------------------------------------------------------
// The chunk sizes accepted: the page's two entry points default to 64 (the CUDA chunkwise one) and
// 128 (the fully batched torch one).  The chunked form computes the same function for every chunk
// size, up to rounding, so both run the same 64-token kernels.
static bool prefill_chunk_size_ok(int chunk_size) { return chunk_size == 64 || chunk_size == 128; }

extern "C" size_t gdn_prefill_workspace_size(int num_seqs, int64_t T, int Hk, int Hv, int K, int V,
                                             int chunk_size) {
    if (num_seqs <= 0 || T < 0 || Hk < 1 || Hv < 1 || Hv % Hk != 0 || K != 128 || V != 128 ||
        !prefill_chunk_size_ok(chunk_size) || T >= (1LL << 31) - 64)
        return 0;
    return gdn::prefill_workspace_bytes(T, num_seqs, Hv);
}

// gdn_prefill_chunked, gdn_prefill_chunked_f16 and comba_prefill_chunked: the same checks and
// launch, the token arrays (q, k, v, a, b, out) in bf16 or in IEEE binary16; for Comba (a, b, A_log,
// dt_bias unused) the read keys, log decays and betas of CombaIn instead.
struct CombaIn {
    const void* p;
    const void* beta;
    const float* g;
};
namespace {
// The prefill kernels' wait limit (gdn_prefill_set_wait_limit): 0 means the built-in limits.
std::atomic<uint32_t> g_prefill_wait_polls{0};
constexpr uint32_t kPrefillBusyPolls = 1u << 26;   // seconds of busy polling
constexpr uint32_t kPrefillSleepPolls = 1u << 22;  // polls with a 1 us suspend hint: seconds
}  // namespace

extern "C" void gdn_prefill_set_wait_limit(uint32_t polls) {
    g_prefill_wait_polls.store(polls, std::memory_order_relaxed);
}

static gdn_status prefill_entry(const char* fn, bool f16, const void* q, const void* k, const void* v,
                                const void* a, const void* b, const float* A_log, const float* dt_bias,
                                float* state_pool, int pool_size, const int64_t* cache_indices,
                                const int64_t* cu_seqlens, int num_seqs, int64_t T, int Hk, int Hv, int K,
                                int V, int chunk_size, float scale, void* out, void* workspace,
                                size_t workspace_bytes, int32_t* dev_status, gdn_stream_t stream,
                                const CombaIn* cb = nullptr) {
    REQUIRE(num_seqs >= 0 && T >= 0 && pool_size >= 0 && Hk >= 1 && Hv >= 1 && K >= 1 && V >= 1,
            GDN_ERR_INVALID_ARG, "%s: sizes must be num_seqs, T, pool_size >= 0 and Hk, Hv, K, V >= 1", fn);
    REQUIRE(Hv % Hk == 0, GDN_ERR_INVALID_ARG, "%s: Hv (%d) must be a multiple of Hk (%d)", fn, Hv, Hk);
    REQUIRE(K == 128 && V == 128, GDN_ERR_UNSUPPORTED, "%s: K and V must be 128 (got K=%d V=%d)", fn, K, V);
    REQUIRE(prefill_chunk_size_ok(chunk_size), GDN_ERR_UNSUPPORTED, "%s: chunk_size must be 64 or 128 (got %d)",
            fn, chunk_size);
    if (num_seqs == 0) return GDN_OK;
    REQUIRE(cache_indices && cu_seqlens && dev_status && state_pool && (cb || (A_log && dt_bias)),
            GDN_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (cb) {
        REQUIRE(T == 0 || (q && k && v && cb->p && cb->beta && cb->g && out), GDN_ERR_INVALID_ARG,
                "%s: null token pointer", fn);
        REQUIRE(aligned(cb->p, 16) && aligned(cb->beta, 2) && aligned(cb->g, 4), GDN_ERR_INVALID_ARG,
                "%s: misaligned argument (p 16 bytes, beta 2, g 4)", fn);
    } else {
        REQUIRE(T == 0 || (q && k && v && a && b && out), GDN_ERR_INVALID_ARG, "%s: null token pointer", fn);
        REQUIRE(aligned(a, 2) && aligned(b, 2) && aligned(A_log, 4) && aligned(dt_bias, 4), GDN_ERR_INVALID_ARG,
                "%s: misaligned argument", fn);
    }
    REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(out, 16) && aligned(state_pool, 16),
            GDN_ERR_INVALID_ARG, "%s: q, k, v, out and state_pool must be 16-byte aligned", fn);
    REQUIRE(aligned(dev_status, 4) && aligned(cache_indices, 8) && aligned(cu_seqlens, 8),
            GDN_ERR_INVALID_ARG, "%s: misaligned argument", fn);
    const size_t obytes = size_t(T) * Hv * V * 2, pbytes = size_t(pool_size) * Hv * V * K * 4;
    REQUIRE(!any_overlap(out, obytes, state_pool, pbytes), GDN_ERR_INVALID_ARG, "%s: out overlaps state_pool",
            fn);
    REQUIRE((long long)(num_seqs + 2 * gdn::kPfMaxSplits) * Hv < (1LL << 31) && T < (1LL << 31) - 64 &&
                gdn::prefill_chunk_cap(T, num_seqs) * Hv < (1LL << 31),
            GDN_ERR_UNSUPPORTED, "%s: grid or token count too large", fn);
    const gdn::PrefillLayout lay = gdn::prefill_layout(T, num_seqs, Hv);
    REQUIRE(workspace && workspace_bytes >= lay.bytes_min, GDN_ERR_INVALID_ARG,
            "%s: workspace of %zu bytes given, %zu needed", fn, workspace ? workspace_bytes : 0, lay.bytes_min);
    REQUIRE(aligned(workspace, 256), GDN_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
    const size_t ws_used = gdn::prefill_splits(lay, workspace_bytes, num_seqs) ? lay.bytes_full : lay.bytes_min;
    REQUIRE(!any_overlap(workspace, ws_used, out, obytes) && !any_overlap(workspace, ws_used, state_pool, pbytes),
            GDN_ERR_INVALID_ARG, "%s: workspace overlaps out or state_pool", fn);

    gdn::PrefillArgs p;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(b);
    p.A_log = A_log;
    p.dt_bias = dt_bias;
    p.p = cb ? static_cast<const uint16_t*>(cb->p) : nullptr;
    p.g_log = cb ? cb->g : nullptr;
    p.beta_in = cb ? static_cast<const uint16_t*>(cb->beta) : nullptr;
    p.state_pool = state_pool;
    p.cache_indices = cache_indices;
    p.cu_seqlens = cu_seqlens;
    p.out = static_cast<uint16_t*>(out);
    p.status = dev_status;
    p.T = T;
    p.pool_size = pool_size;
    p.num_seqs = num_seqs;
    p.Hk = Hk;
    p.Hv = Hv;
    p.scale = scale;
    p.eps = 1e-6f;
    const uint32_t polls = g_prefill_wait_polls.load(std::memory_order_relaxed);
    p.wait_polls = polls ? polls : kPrefillBusyPolls;
    p.sleep_polls = polls ? polls : kPrefillSleepPolls;
    const cudaError_t e =
        gdn::launch_prefill(p, workspace, workspace_bytes, static_cast<cudaStream_t>(stream), f16, cb != nullptr);
    if (e != cudaSuccess)
        return fail(GDN_ERR_CUDA, "%s: launch failed (TMA descriptors or kernel): %s", fn, cudaGetErrorString(e));
    g_last_error[0] = '\0';
    return GDN_OK;
}

extern "C" gdn_status gdn_prefill_chunked(const void* q, const void* k, const void* v, const void* a,
                                          const void* b, const float* A_log, const float* dt_bias,
                                          float* state_pool, int pool_size,
                                          const int64_t* cache_indices, const int64_t* cu_seqlens,
                                          int num_seqs, int64_t T, int Hk, int Hv, int K, int V,
                                          int chunk_size, float scale, void* out, void* workspace,
                                          size_t workspace_bytes, int32_t* dev_status,
                                          gdn_stream_t stream) {
    return prefill_entry("gdn_prefill_chunked", false, q, k, v, a, b, A_log, dt_bias, state_pool, pool_size,
                         cache_indices, cu_seqlens, num_seqs, T, Hk, Hv, K, V, chunk_size, scale, out,
                         workspace, workspace_bytes, dev_status, stream);
}

extern "C" gdn_status gdn_prefill_chunked_f16(const void* q, const void* k, const void* v, const void* a,
                                              const void* b, const float* A_log, const float* dt_bias,
                                              float* state_pool, int pool_size,
                                              const int64_t* cache_indices, const int64_t* cu_seqlens,
                                              int num_seqs, int64_t T, int Hk, int Hv, int K, int V,
                                              int chunk_size, float scale, void* out, void* workspace,
                                              size_t workspace_bytes, int32_t* dev_status,
                                              gdn_stream_t stream) {
    return prefill_entry("gdn_prefill_chunked_f16", true, q, k, v, a, b, A_log, dt_bias, state_pool, pool_size,
                         cache_indices, cu_seqlens, num_seqs, T, Hk, Hv, K, V, chunk_size, scale, out,
                         workspace, workspace_bytes, dev_status, stream);
}

extern "C" gdn_status comba_prefill_chunked(const void* q, const void* k, const void* v, const void* p,
                                            const void* beta, const float* g, float* state_pool, int pool_size,
                                            const int64_t* cache_indices, const int64_t* cu_seqlens,
                                            int num_seqs, int64_t T, int H, int K, int V, int chunk_size,
                                            float scale, void* out, void* workspace, size_t workspace_bytes,
                                            int32_t* dev_status, gdn_stream_t stream) {
    const CombaIn cb{p, beta, g};
    return prefill_entry("comba_prefill_chunked", false, q, k, v, nullptr, nullptr, nullptr, nullptr, state_pool,
                         pool_size, cache_indices, cu_seqlens, num_seqs, T, H, H, K, V, chunk_size, scale, out,
                         workspace, workspace_bytes, dev_status, stream, &cb);
}


// ------------------------------------------------------------------------------------------------
extern "C" gdn_status gdn_window_fused(float* state, const float* hist, float* hist_out,
                                       const float* qkv, const float* alpha, const float* beta,
                                       const float* z, const float* conv_w, const float* dt,
                                       const float* ssm_a, const float* gamma, float* y, int N,
                                       int h_k, int h_v, int ntok, unsigned commit, float eps,
                                       gdn_stream_t stream) {
    REQUIRE(N >= 0 && h_k >= 1 && h_v >= 1, GDN_ERR_INVALID_ARG,
            "gdn_window_fused: sizes must be N >= 0 and h_k, h_v >= 1 (got N=%d h_k=%d h_v=%d)", N, h_k,
            h_v);
    REQUIRE(ntok >= 1 && ntok <= gdn::kWinMaxTok, GDN_ERR_UNSUPPORTED,
            "gdn_window_fused: ntok must be in [1, %d] (got %d)", gdn::kWinMaxTok, ntok);
    REQUIRE(h_k <= h_v, GDN_ERR_UNSUPPORTED,
            "gdn_window_fused: h_k (%d) must not exceed h_v (%d)", h_k, h_v);
    int commit_at = -1;
    if (commit == 0u) commit_at = 0;
    else if (commit == 1u) commit_at = ntok;
    else if ((commit >> 8) == 1u && (commit & 0xffu) >= 1u && int(commit & 0xffu) <= ntok)
        commit_at = int(commit & 0xffu);
    REQUIRE(commit_at >= 0, GDN_ERR_INVALID_ARG,
            "gdn_window_fused: commit must be 0, 1 or 0x100|k with 1 <= k <= ntok (got 0x%x)", commit);
    if (N == 0) return GDN_OK;
    REQUIRE(state && hist && hist_out && qkv && alpha && beta && z && conv_w && dt && ssm_a && gamma &&
                y, GDN_ERR_INVALID_ARG, "gdn_window_fused: null pointer");
    const size_t C = size_t(2 * h_k + h_v) * gdn::kWinD;
    const size_t hbytes = size_t(N) * C * 3 * sizeof(float);
    REQUIRE(!any_overlap(hist, hbytes, hist_out, hbytes), GDN_ERR_INVALID_ARG,
            "gdn_window_fused: hist_out must not overlap hist (the q/k history is read by several heads)");
    const size_t sbytes = size_t(N) * gdn::kWinD * h_v * gdn::kWinD * sizeof(float);
    const size_t ybytes = size_t(N) * ntok * h_v * gdn::kWinD * sizeof(float);
    REQUIRE(!any_overlap(y, ybytes, state, sbytes) && !any_overlap(y, ybytes, hist_out, hbytes) &&
                !any_overlap(state, sbytes, hist_out, hbytes),
            GDN_ERR_INVALID_ARG, "gdn_window_fused: y, state and hist_out must not overlap");
    REQUIRE(aligned(state, 16) && aligned(conv_w, 16), GDN_ERR_INVALID_ARG,
            "gdn_window_fused: state and conv_w must be 16-byte aligned");
    REQUIRE(aligned(hist, 4) && aligned(hist_out, 4) && aligned(qkv, 4) && aligned(alpha, 4) &&
                aligned(beta, 4) && aligned(z, 4) && aligned(dt, 4) && aligned(ssm_a, 4) &&
                aligned(gamma, 4) && aligned(y, 4),
            GDN_ERR_INVALID_ARG, "gdn_window_fused: float arrays must be 4-byte aligned");
    REQUIRE(1LL * N * h_v < (1LL << 31), GDN_ERR_UNSUPPORTED, "gdn_window_fused: grid too large");

    gdn::WindowArgs a;
    a.state = state;
    a.hist = hist;
    a.hist_out = hist_out;
    a.qkv = qkv;
    a.alpha = alpha;
    a.beta = beta;
    a.z = z;
    a.conv_w = conv_w;
    a.dt = dt;
    a.ssm_a = ssm_a;
    a.gamma = gamma;
    a.y = y;
    a.h_k = h_k;
    a.h_v = h_v;
    a.ntok = ntok;
    a.commit_at = commit_at;
    a.eps = eps;
    const cudaError_t e = gdn::launch_window(a, N, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return fail(GDN_ERR_CUDA, "gdn_window_fused: launch failed: %s", cudaGetErrorString(e));
    g_last_error[0] = '\0';
    return GDN_OK;
}

// ------------------------------------------------------------------------------------------------
// gdn_prefill_chunked_noalloc: the prefill for callers that cannot allocate device memory
// themselves (a host framework whose allocator owns all device memory, or code running where a
// cudaMalloc is not allowed).  Its workspace is a file-scope device array of fixed size, which
// every GPU that loads this library holds until the process exits.  Host code sees only a
// host-side stand-in for the array, so its device address is looked up once per device, with that
// device current, and handed to the kernels.
namespace {

constexpr size_t kNoallocScratchBytes = size_t(64) << 20;  // 64 MiB
static __device__ __align__(256) uint8_t g_prefill_scratch[kNoallocScratchBytes];

constexpr int kNoallocMaxDevices = 64;
void* g_scratch_ptr[kNoallocMaxDevices];    // the array's device address on each device
std::atomic<int> g_scratch_ready[kNoallocMaxDevices];
std::mutex g_scratch_mutex;

}  // namespace

extern "C" gdn_status gdn_prefill_chunked_noalloc(const void* q, const void* k, const void* v, const void* a,
                                                  const void* b, const float* A_log, const float* dt_bias,
                                                  float* state_pool, int pool_size,
                                                  const int64_t* cache_indices, const int64_t* cu_seqlens,
                                                  int num_seqs, int64_t T, int Hk, int Hv, int K, int V,
                                                  int chunk_size, float scale, void* out,
                                                  int32_t* dev_status, gdn_stream_t stream) {
    // the scratch must hold the records; long sequences are split only when it also holds the
    // split scratch
    const size_t full = gdn_prefill_workspace_size(num_seqs, T, Hk, Hv, K, V, chunk_size);
    const size_t need = full == 0 ? 0 : gdn::prefill_layout(T, num_seqs, Hv).bytes_min;
    REQUIRE(need <= kNoallocScratchBytes, GDN_ERR_UNSUPPORTED,
            "gdn_prefill_chunked_noalloc: these sizes need %zu bytes of workspace (%zu without splitting "
            "long sequences); the library's static scratch holds %zu (use gdn_prefill_chunked with a "
            "caller-owned workspace)",
            full, need, kNoallocScratchBytes);
    if (num_seqs == 0)  // nothing runs; the scratch is not needed
        return gdn_prefill_chunked(q, k, v, a, b, A_log, dt_bias, state_pool, pool_size, cache_indices,
                                   cu_seqlens, num_seqs, T, Hk, Hv, K, V, chunk_size, scale, out, nullptr, 0,
                                   dev_status, stream);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return fail(GDN_ERR_CUDA, "gdn_prefill_chunked_noalloc: cudaGetDevice: %s", cudaGetErrorString(e));
    REQUIRE(dev >= 0 && dev < kNoallocMaxDevices, GDN_ERR_UNSUPPORTED,
            "gdn_prefill_chunked_noalloc: device %d beyond the %d supported", dev, kNoallocMaxDevices);
    if (!g_scratch_ready[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_scratch_mutex);
        if (!g_scratch_ready[dev].load(std::memory_order_relaxed)) {
            void* p = nullptr;
            e = cudaGetSymbolAddress(&p, g_prefill_scratch);
            if (e != cudaSuccess || p == nullptr)
                return fail(GDN_ERR_CUDA, "gdn_prefill_chunked_noalloc: cudaGetSymbolAddress of the scratch: %s",
                            cudaGetErrorString(e));
            g_scratch_ptr[dev] = p;
            g_scratch_ready[dev].store(1, std::memory_order_release);
        }
    }
    return gdn_prefill_chunked(q, k, v, a, b, A_log, dt_bias, state_pool, pool_size, cache_indices, cu_seqlens,
                               num_seqs, T, Hk, Hv, K, V, chunk_size, scale, out, g_scratch_ptr[dev],
                               kNoallocScratchBytes, dev_status, stream);
}

// ------------------------------------------------------------------------------------------------
// the paged attention cache, attention over it, and draft verification
namespace {
std::atomic<uint32_t> g_attn_wait_polls{0};  // attn_set_wait_limit
}  // namespace

extern "C" void attn_set_wait_limit(uint32_t polls) { g_attn_wait_polls.store(polls, std::memory_order_relaxed); }

static bool attn_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

// What attn_cache_write, attn_cache_read and attn_paged ask of their cache.
static gdn_status cache_check(const char* fn, const void* kc, const void* vc, const float* ks, const float* vs,
                              gdn_dtype cache_dtype, gdn_dtype dtype, int64_t num_pages, int page_size, int Hkv,
                              int D, const int32_t* dev_status, size_t* bytes) {
    REQUIRE(dtype == GDN_BF16 || dtype == GDN_F16, GDN_ERR_INVALID_ARG, "%s: dtype must be GDN_BF16 or GDN_F16", fn);
    REQUIRE(cache_dtype == dtype || cache_dtype == GDN_E4M3, GDN_ERR_INVALID_ARG,
            "%s: cache_dtype must be dtype or GDN_E4M3", fn);
    REQUIRE(attn_dim_ok(D), GDN_ERR_UNSUPPORTED, "%s: D must be 64, 128 or 256 (got %d)", fn, D);
    REQUIRE(Hkv <= 65535, GDN_ERR_UNSUPPORTED, "%s: at most 65535 heads (got %d)", fn, Hkv);
    REQUIRE(kc && vc && dev_status, GDN_ERR_INVALID_ARG, "%s: null pointer", fn);
    REQUIRE(aligned(kc, 16) && aligned(vc, 16) && aligned(dev_status, 4), GDN_ERR_INVALID_ARG,
            "%s: caches must be 16-byte aligned", fn);
    if (cache_dtype == GDN_E4M3)
        REQUIRE(ks && vs && aligned(ks, 4) && aligned(vs, 4), GDN_ERR_INVALID_ARG,
                "%s: an 8-bit cache needs k_scale and v_scale", fn);
    else
        REQUIRE(!ks && !vs, GDN_ERR_INVALID_ARG, "%s: a cache of dtype has no scales", fn);
    const long long rows_per_page = static_cast<long long>(Hkv) * page_size;
    REQUIRE(num_pages <= (1LL << 52) / (rows_per_page * D), GDN_ERR_UNSUPPORTED, "%s: cache too large", fn);
    *bytes = static_cast<size_t>(num_pages) * rows_per_page * D * (cache_dtype == GDN_E4M3 ? 1 : 2);
    return GDN_OK;
}

extern "C" gdn_status attn_cache_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                                       gdn_dtype dtype, const int64_t* slots, int64_t T, void* k_cache,
                                       void* v_cache, float* k_scale, float* v_scale, gdn_dtype cache_dtype,
                                       int64_t num_pages, int page_size, int Hkv, int D, int32_t* dev_status,
                                       gdn_stream_t stream) {
    const char* fn = "attn_cache_write";
    REQUIRE(T >= 0 && num_pages >= 0 && page_size >= 1 && Hkv >= 1, GDN_ERR_INVALID_ARG,
            "%s: sizes must be T, num_pages >= 0 and page_size, Hkv >= 1", fn);
    if (T == 0) return GDN_OK;
    size_t cb = 0;
    const gdn_status s = cache_check(fn, k_cache, v_cache, k_scale, v_scale, cache_dtype, dtype, num_pages, page_size,
                                     Hkv, D, dev_status, &cb);
    if (s != GDN_OK) return s;
    REQUIRE(k && v && slots, GDN_ERR_INVALID_ARG, "%s: null pointer", fn);
    const long long row = static_cast<long long>(Hkv) * D;
    REQUIRE(k_stride >= row && v_stride >= row && k_stride % 8 == 0 && v_stride % 8 == 0, GDN_ERR_INVALID_ARG,
            "%s: token strides must be multiples of 8 and at least Hkv * D", fn);
    REQUIRE(aligned(k, 16) && aligned(v, 16) && aligned(slots, 8), GDN_ERR_INVALID_ARG,
            "%s: k and v must be 16-byte aligned", fn);
    REQUIRE(T < (1LL << 31) && k_stride < (1LL << 31) && v_stride < (1LL << 31), GDN_ERR_UNSUPPORTED,
            "%s: T and the strides must be below 2^31", fn);
    const size_t kb = (static_cast<size_t>(T - 1) * k_stride + row) * 2, vb = (static_cast<size_t>(T - 1) * v_stride + row) * 2;
    REQUIRE(!any_overlap(k_cache, cb, v_cache, cb) && !any_overlap(k, kb, k_cache, cb) && !any_overlap(k, kb, v_cache, cb) &&
                !any_overlap(v, vb, k_cache, cb) && !any_overlap(v, vb, v_cache, cb),
            GDN_ERR_INVALID_ARG, "%s: the caches overlap each other or the sources", fn);
    const size_t sb = k_scale ? static_cast<size_t>(num_pages) * Hkv * page_size * 4 : 0;
    REQUIRE(!any_overlap(k_scale, sb, v_scale, sb), GDN_ERR_INVALID_ARG, "%s: k_scale and v_scale overlap", fn);
    gdn::CacheMoveArgs a;
    std::memset(&a, 0, sizeof(a));
    a.k_in = static_cast<const uint16_t*>(k);
    a.v_in = static_cast<const uint16_t*>(v);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.kc = k_cache;
    a.vc = v_cache;
    a.ks = k_scale;
    a.vs = v_scale;
    a.slots = slots;
    a.status = dev_status;
    a.T = T;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.H = Hkv;
    gdn::launch_cache_write(a, D, dtype == GDN_F16, cache_dtype == GDN_E4M3, static_cast<cudaStream_t>(stream));
    return launched(fn);
}

extern "C" gdn_status attn_cache_read(const void* k_cache, const void* v_cache, const float* k_scale,
                                      const float* v_scale, gdn_dtype cache_dtype, int64_t num_pages, int page_size,
                                      const int64_t* page_table, int max_pages, const int64_t* cu_seqlens,
                                      int num_seqs, int64_t T, int Hkv, int D, void* k, void* v, gdn_dtype dtype,
                                      int32_t* dev_status, gdn_stream_t stream) {
    const char* fn = "attn_cache_read";
    REQUIRE(T >= 0 && num_seqs >= 0 && num_pages >= 0 && max_pages >= 0 && page_size >= 1 && Hkv >= 1,
            GDN_ERR_INVALID_ARG, "%s: sizes must be T, num_seqs, num_pages, max_pages >= 0 and page_size, Hkv >= 1", fn);
    if (T == 0 || num_seqs == 0) return GDN_OK;
    size_t cb = 0;
    const gdn_status s = cache_check(fn, k_cache, v_cache, k_scale, v_scale, cache_dtype, dtype, num_pages, page_size,
                                     Hkv, D, dev_status, &cb);
    if (s != GDN_OK) return s;
    REQUIRE(k && v && cu_seqlens && (page_table || max_pages == 0), GDN_ERR_INVALID_ARG, "%s: null pointer", fn);
    REQUIRE(aligned(k, 16) && aligned(v, 16) && aligned(cu_seqlens, 8) && aligned(page_table, 8), GDN_ERR_INVALID_ARG,
            "%s: k and v must be 16-byte aligned", fn);
    REQUIRE(T < (1LL << 31), GDN_ERR_UNSUPPORTED, "%s: T must be below 2^31", fn);
    const size_t ob = static_cast<size_t>(T) * Hkv * D * 2;
    REQUIRE(!any_overlap(k, ob, v, ob) && !any_overlap(k, ob, k_cache, cb) && !any_overlap(k, ob, v_cache, cb) &&
                !any_overlap(v, ob, k_cache, cb) && !any_overlap(v, ob, v_cache, cb),
            GDN_ERR_INVALID_ARG, "%s: the outputs overlap each other or the caches", fn);
    gdn::CacheMoveArgs a;
    std::memset(&a, 0, sizeof(a));
    a.k_out = static_cast<uint16_t*>(k);
    a.v_out = static_cast<uint16_t*>(v);
    a.kc = const_cast<void*>(k_cache);
    a.vc = const_cast<void*>(v_cache);
    a.ks = const_cast<float*>(k_scale);
    a.vs = const_cast<float*>(v_scale);
    a.table = page_table;
    a.cu = cu_seqlens;
    a.status = dev_status;
    a.T = T;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.num_seqs = num_seqs;
    a.H = Hkv;
    gdn::launch_cache_read(a, D, dtype == GDN_F16, cache_dtype == GDN_E4M3, static_cast<cudaStream_t>(stream));
    return launched(fn);
}

extern "C" size_t attn_paged_workspace_size(int D) { return attn_dim_ok(D) ? gdn::attn_workspace_bytes(D) : 0; }

extern "C" gdn_status attn_paged(const void* q, int64_t q_stride, gdn_dtype dtype, const void* k_cache,
                                 const void* v_cache, const float* k_scale, const float* v_scale,
                                 gdn_dtype cache_dtype, int64_t num_pages, int page_size, const int64_t* page_table,
                                 int max_pages, const int64_t* kv_lens, const int64_t* cu_seqlens, int num_seqs,
                                 int64_t T, int64_t max_q, int Hq, int Hkv, int D, float scale, void* out, float* lse,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_status, gdn_stream_t stream) {
    const char* fn = "attn_paged";
    REQUIRE(T >= 0 && num_seqs >= 0 && num_pages >= 0 && max_pages >= 0 && max_q >= 0 && page_size >= 1 && Hq >= 1 &&
                Hkv >= 1,
            GDN_ERR_INVALID_ARG,
            "%s: sizes must be T, max_q, num_seqs, num_pages, max_pages >= 0 and page_size, Hq, Hkv >= 1", fn);
    REQUIRE(Hq % Hkv == 0, GDN_ERR_INVALID_ARG, "%s: Hq (%d) must be a multiple of Hkv (%d)", fn, Hq, Hkv);
    REQUIRE(Hq / Hkv <= 128, GDN_ERR_UNSUPPORTED, "%s: Hq / Hkv must be at most 128 (got %d)", fn, Hq / Hkv);
    if (T == 0 || num_seqs == 0) return GDN_OK;
    size_t cb = 0;
    const gdn_status s = cache_check(fn, k_cache, v_cache, k_scale, v_scale, cache_dtype, dtype, num_pages, page_size,
                                     Hkv, D, dev_status, &cb);
    if (s != GDN_OK) return s;
    REQUIRE(q && out && kv_lens && cu_seqlens && (page_table || max_pages == 0), GDN_ERR_INVALID_ARG,
            "%s: null pointer", fn);
    REQUIRE(q_stride >= static_cast<int64_t>(Hq) * D && q_stride % 8 == 0 && q_stride < (1LL << 31), GDN_ERR_INVALID_ARG,
            "%s: q_stride must be a multiple of 8, at least Hq * D and below 2^31", fn);
    REQUIRE(aligned(q, 16) && aligned(out, 16) && aligned(lse, 4) && aligned(kv_lens, 8) && aligned(cu_seqlens, 8) &&
                aligned(page_table, 8),
            GDN_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", fn);
    REQUIRE(T < (1LL << 30) && static_cast<long long>(max_pages) * page_size < (1LL << 31), GDN_ERR_UNSUPPORTED,
            "%s: T must be below 2^30 and max_pages * page_size below 2^31", fn);
    const size_t need = gdn::attn_workspace_bytes(D);
    REQUIRE(workspace && workspace_bytes >= need, GDN_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed (got %zu)", fn,
            need, workspace ? workspace_bytes : size_t(0));
    REQUIRE(aligned(workspace, 16), GDN_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
    const size_t ob = static_cast<size_t>(T) * Hq * D * 2, lb = lse ? static_cast<size_t>(T) * Hq * 4 : 0;
    const size_t qb = (static_cast<size_t>(T - 1) * q_stride + static_cast<size_t>(Hq) * D) * 2;
    REQUIRE(!any_overlap(out, ob, q, qb) && !any_overlap(out, ob, workspace, need) && !any_overlap(out, ob, lse, lb) &&
                !any_overlap(out, ob, k_cache, cb) && !any_overlap(out, ob, v_cache, cb) &&
                !any_overlap(lse, lb, workspace, need) && !any_overlap(workspace, need, q, qb) &&
                !any_overlap(workspace, need, k_cache, cb) && !any_overlap(workspace, need, v_cache, cb),
            GDN_ERR_INVALID_ARG, "%s: out, lse or workspace overlaps another buffer", fn);
    gdn::AttnArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.kc = k_cache;
    a.vc = v_cache;
    a.ks = k_scale;
    a.vs = v_scale;
    a.table = page_table;
    a.kv_lens = kv_lens;
    a.cu = cu_seqlens;
    a.out = out;
    a.lse = lse;
    a.status = dev_status;
    a.T = T;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.num_seqs = num_seqs;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.f16 = dtype == GDN_F16;
    a.scale_log2 = scale * 1.44269504088896340736f;
    int sh = 0;
    while ((1LL << sh) < page_size) ++sh;
    a.page_mul = static_cast<uint32_t>(((1ULL << (31 + sh)) + page_size - 1) / page_size);
    a.page_shift = 31 + sh;
    a.polls = g_attn_wait_polls.load(std::memory_order_relaxed);
    const cudaError_t e =
        gdn::launch_attn(a, workspace, D, cache_dtype == GDN_E4M3, static_cast<int>(max_q < T ? max_q : T), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    return launched(fn);
}

extern "C" gdn_status draft_verify(const float* target_p, const float* draft_p, const int64_t* drafts,
                                   const int64_t* num_drafts, const float* u_accept, const float* u_sample, int N,
                                   int T, int V, int64_t* accepted, int64_t* tokens, int32_t* dev_status,
                                   gdn_stream_t stream) {
    const char* fn = "draft_verify";
    REQUIRE(N >= 0 && T >= 0 && V >= 1, GDN_ERR_INVALID_ARG, "%s: sizes must be N, T >= 0 and V >= 1", fn);
    REQUIRE(V <= (1 << 20), GDN_ERR_UNSUPPORTED, "%s: V must be at most 2^20 (got %d)", fn, V);
    REQUIRE(N < (1 << 28), GDN_ERR_UNSUPPORTED, "%s: N must be below 2^28", fn);
    if (N == 0) return GDN_OK;
    REQUIRE(target_p && u_sample && accepted && tokens && dev_status && (T == 0 || (draft_p && drafts && u_accept)),
            GDN_ERR_INVALID_ARG, "%s: null pointer", fn);
    REQUIRE(aligned(target_p, 4) && aligned(draft_p, 4) && aligned(drafts, 8) && aligned(num_drafts, 8) &&
                aligned(u_accept, 4) && aligned(u_sample, 4) && aligned(accepted, 8) && aligned(tokens, 8) &&
                aligned(dev_status, 4),
            GDN_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    const size_t tb = static_cast<size_t>(N) * (T + 1) * 8;
    REQUIRE(!any_overlap(tokens, tb, drafts, static_cast<size_t>(N) * T * 8) &&
                !any_overlap(tokens, tb, accepted, static_cast<size_t>(N) * 8),
            GDN_ERR_INVALID_ARG, "%s: tokens overlaps drafts or accepted", fn);
    gdn::VerifyArgs a;
    a.target = target_p;
    a.draft = draft_p;
    a.drafts = drafts;
    a.num_drafts = num_drafts;
    a.u_accept = u_accept;
    a.u_sample = u_sample;
    a.accepted = accepted;
    a.tokens = tokens;
    a.status = dev_status;
    a.N = N;
    a.T = T;
    a.V = V;
    const cudaError_t e = gdn::launch_verify(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    return launched(fn);
}

// ------------------------------------------------------------------------------------------------
// what stands between the matrix products: rotation with the append, short convolution, state space scan, norm
extern "C" gdn_status attn_cache_append(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                        int64_t v_stride, gdn_dtype dtype, const float* rotation, int64_t max_positions,
                                        int rotary_dim, int neighbours, const int64_t* positions, const int64_t* slots,
                                        int64_t T, void* q_out, int64_t q_out_stride, void* k_cache, void* v_cache,
                                        float* k_scale, float* v_scale, gdn_dtype cache_dtype, int64_t num_pages,
                                        int page_size, int Hq, int Hkv, int D, int32_t* dev_status, gdn_stream_t stream) {
    const char* fn = "attn_cache_append";
    REQUIRE(T >= 0 && num_pages >= 0 && max_positions >= 0 && Hq >= 0 && page_size >= 1 && Hkv >= 1, GDN_ERR_INVALID_ARG,
            "%s: sizes must be T, num_pages, max_positions, Hq >= 0 and page_size, Hkv >= 1", fn);
    if (T == 0) return GDN_OK;
    size_t cb = 0;
    const gdn_status s = cache_check(fn, k_cache, v_cache, k_scale, v_scale, cache_dtype, dtype, num_pages, page_size,
                                     Hkv, D, dev_status, &cb);
    if (s != GDN_OK) return s;
    REQUIRE(Hq <= 65535, GDN_ERR_UNSUPPORTED, "%s: at most 65535 heads (got %d)", fn, Hq);
    REQUIRE(rotary_dim >= 16 && rotary_dim <= D && rotary_dim % 16 == 0, GDN_ERR_UNSUPPORTED,
            "%s: rotary_dim must be a multiple of 16 between 16 and D (got %d)", fn, rotary_dim);
    REQUIRE(k && v && slots && positions && rotation && (Hq == 0 || (q && q_out)), GDN_ERR_INVALID_ARG, "%s: null pointer", fn);
    const long long row = static_cast<long long>(Hkv) * D, qrow = static_cast<long long>(Hq) * D;
    REQUIRE(k_stride >= row && v_stride >= row && k_stride % 8 == 0 && v_stride % 8 == 0 &&
                (Hq == 0 || (q_stride >= qrow && q_out_stride >= qrow && q_stride % 8 == 0 && q_out_stride % 8 == 0)),
            GDN_ERR_INVALID_ARG, "%s: token strides must be multiples of 8 and at least the heads' width", fn);
    REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(q_out, 16) && aligned(rotation, 16) &&
                aligned(slots, 8) && aligned(positions, 8),
            GDN_ERR_INVALID_ARG, "%s: q, k, v, q_out and rotation must be 16-byte aligned", fn);
    REQUIRE(T < (1LL << 31) && k_stride < (1LL << 31) && v_stride < (1LL << 31) &&
                (Hq == 0 || (q_stride < (1LL << 31) && q_out_stride < (1LL << 31))),
            GDN_ERR_UNSUPPORTED, "%s: T and the strides must be below 2^31", fn);
    REQUIRE(max_positions <= (1LL << 52) / rotary_dim, GDN_ERR_UNSUPPORTED, "%s: max_positions too large", fn);
    REQUIRE((T / 8 + 1) * ((Hq + 2LL * Hkv) / 4 + 3) < (1LL << 31), GDN_ERR_UNSUPPORTED, "%s: too many tokens and heads for one call", fn);
    const size_t kb = (static_cast<size_t>(T - 1) * k_stride + row) * 2, vb = (static_cast<size_t>(T - 1) * v_stride + row) * 2;
    const size_t qb = Hq ? (static_cast<size_t>(T - 1) * q_stride + qrow) * 2 : 0;
    const size_t ob = Hq ? (static_cast<size_t>(T - 1) * q_out_stride + qrow) * 2 : 0;
    REQUIRE(!any_overlap(k_cache, cb, v_cache, cb) && !any_overlap(k, kb, k_cache, cb) && !any_overlap(k, kb, v_cache, cb) &&
                !any_overlap(v, vb, k_cache, cb) && !any_overlap(v, vb, v_cache, cb) && !any_overlap(q, qb, k_cache, cb) &&
                !any_overlap(q, qb, v_cache, cb) && !any_overlap(q_out, ob, k_cache, cb) && !any_overlap(q_out, ob, v_cache, cb),
            GDN_ERR_INVALID_ARG, "%s: the caches overlap each other, the sources or q_out", fn);
    const size_t rb = static_cast<size_t>(max_positions) * rotary_dim * 4;
    // q_out may be q itself; then its rows may stand among the rows of k and v, as those of a fused projection do
    const bool in_place = Hq > 0 && q_out == q && q_out_stride == q_stride;
    auto apart = [&](const void* p, size_t bytes, int64_t stride) {
        if (!any_overlap(q_out, ob, p, bytes)) return true;
        if (!in_place || stride != q_stride) return false;
        const long long d = (static_cast<long long>(reinterpret_cast<uintptr_t>(p)) - static_cast<long long>(reinterpret_cast<uintptr_t>(q))) / 2 % q_stride;
        const long long behind = d < 0 ? d + q_stride : d;
        return behind >= qrow && behind + row <= q_stride;
    };
    REQUIRE((in_place || !any_overlap(q_out, ob, q, qb)) && apart(k, kb, k_stride) && apart(v, vb, v_stride), GDN_ERR_INVALID_ARG,
            "%s: q_out overlaps a source (it may be q itself, with the same stride)", fn);
    REQUIRE(!any_overlap(q_out, ob, rotation, rb) && !any_overlap(k_cache, cb, rotation, rb) && !any_overlap(v_cache, cb, rotation, rb),
            GDN_ERR_INVALID_ARG, "%s: rotation overlaps an output", fn);
    const size_t sb = k_scale ? static_cast<size_t>(num_pages) * Hkv * page_size * 4 : 0;
    REQUIRE(!any_overlap(k_scale, sb, v_scale, sb), GDN_ERR_INVALID_ARG, "%s: k_scale and v_scale overlap", fn);
    for (const float* scale : {k_scale, v_scale})
        REQUIRE(!any_overlap(scale, sb, k_cache, cb) && !any_overlap(scale, sb, v_cache, cb) && !any_overlap(scale, sb, k, kb) &&
                    !any_overlap(scale, sb, v, vb) && !any_overlap(scale, sb, q, qb) && !any_overlap(scale, sb, q_out, ob) &&
                    !any_overlap(scale, sb, rotation, rb),
                GDN_ERR_INVALID_ARG, "%s: a scale overlaps another buffer", fn);
    gdn::AppendArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.q_out_stride = q_out_stride;
    a.rotation = rotation;
    a.positions = positions;
    a.slots = slots;
    a.kc = k_cache;
    a.vc = v_cache;
    a.ks = k_scale;
    a.vs = v_scale;
    a.status = dev_status;
    a.T = T;
    a.num_pages = num_pages;
    a.max_pos = max_positions;
    a.page_size = page_size;
    a.Hq = Hq;
    a.H = Hkv;
    a.turned = rotary_dim;
    gdn::launch_cache_append(a, D, dtype == GDN_F16, cache_dtype == GDN_E4M3, neighbours != 0, static_cast<cudaStream_t>(stream));
    return launched(fn);
}

extern "C" gdn_status short_conv(const void* x, int64_t x_stride, gdn_dtype dtype, const float* weight, const float* bias,
                                 float* hist_pool, int pool_size, const int64_t* cache_indices, const int64_t* cu_seqlens,
                                 int num_seqs, int64_t T, int C, int taps, int silu, void* out0, int c0, void* out1, int c1,
                                 void* out2, int c2, int32_t* dev_status, gdn_stream_t stream) {
    const char* fn = "short_conv";
    REQUIRE(T >= 0 && num_seqs >= 0 && pool_size >= 0 && C >= 1, GDN_ERR_INVALID_ARG,
            "%s: sizes must be T, num_seqs, pool_size >= 0 and C >= 1", fn);
    REQUIRE(dtype == GDN_BF16 || dtype == GDN_F16, GDN_ERR_INVALID_ARG, "%s: dtype must be GDN_BF16 or GDN_F16", fn);
    REQUIRE(taps >= 2 && taps <= 4, GDN_ERR_UNSUPPORTED, "%s: taps must be 2, 3 or 4 (got %d)", fn, taps);
    REQUIRE(c0 >= 1 && c1 >= 0 && c2 >= 0 && (c1 > 0 || c2 == 0) && static_cast<long long>(c0) + c1 + c2 == C, GDN_ERR_INVALID_ARG,
            "%s: the outputs' widths must be positive and add up to C", fn);
    REQUIRE(c0 % 8 == 0 && c1 % 8 == 0 && c2 % 8 == 0, GDN_ERR_UNSUPPORTED, "%s: the outputs' widths must be multiples of 8", fn);
    REQUIRE(C <= (1 << 24) && T < (1LL << 31), GDN_ERR_UNSUPPORTED, "%s: C must be at most 2^24 and T below 2^31", fn);
    if (T == 0 || num_seqs == 0) return GDN_OK;
    REQUIRE(cu_seqlens || T == num_seqs, GDN_ERR_INVALID_ARG, "%s: without cu_seqlens T must be num_seqs", fn);
    REQUIRE(x && weight && hist_pool && cache_indices && dev_status && out0 && (c1 == 0 || out1) && (c2 == 0 || out2),
            GDN_ERR_INVALID_ARG, "%s: null pointer", fn);
    REQUIRE(x_stride >= C && x_stride % 8 == 0 && x_stride < (1LL << 31), GDN_ERR_INVALID_ARG,
            "%s: x_stride must be a multiple of 8, at least C and below 2^31", fn);
    REQUIRE(aligned(x, 16) && aligned(weight, 16) && aligned(bias, 4) && aligned(hist_pool, 16) && aligned(out0, 16) &&
                aligned(out1, 16) && aligned(out2, 16) && aligned(cache_indices, 8) && aligned(cu_seqlens, 8) && aligned(dev_status, 4),
            GDN_ERR_INVALID_ARG, "%s: x, weight, hist_pool and the outputs must be 16-byte aligned", fn);
    const size_t xb = (static_cast<size_t>(T - 1) * x_stride + C) * 2, hb = static_cast<size_t>(pool_size) * C * (taps - 1) * 4;
    const size_t wb = static_cast<size_t>(C) * taps * 4, bb = bias ? static_cast<size_t>(C) * 4 : 0;
    void* const outs[3] = {out0, out1, out2};
    const int widths[3] = {c0, c1, c2};
    REQUIRE(!any_overlap(hist_pool, hb, x, xb) && !any_overlap(hist_pool, hb, weight, wb) && !any_overlap(hist_pool, hb, bias, bb),
            GDN_ERR_INVALID_ARG, "%s: hist_pool overlaps an input", fn);
    for (int i = 0; i < 3; ++i) {
        const size_t ob = static_cast<size_t>(T) * widths[i] * 2;
        REQUIRE(!any_overlap(outs[i], ob, x, xb) && !any_overlap(outs[i], ob, hist_pool, hb) && !any_overlap(outs[i], ob, weight, wb) &&
                    !any_overlap(outs[i], ob, bias, bb),
                GDN_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
        for (int j = 0; j < i; ++j)
            REQUIRE(!any_overlap(outs[i], ob, outs[j], static_cast<size_t>(T) * widths[j] * 2), GDN_ERR_INVALID_ARG,
                    "%s: the outputs overlap", fn);
    }
    gdn::ConvArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = static_cast<const uint16_t*>(x);
    a.x_stride = x_stride;
    a.w = weight;
    a.bias = bias;
    a.hist = hist_pool;
    a.slots = cache_indices;
    a.cu = cu_seqlens;
    for (int i = 0; i < 3; ++i) {
        a.out[i] = static_cast<uint16_t*>(outs[i]);
        a.width[i] = widths[i];
    }
    a.status = dev_status;
    a.T = T;
    a.C = C;
    a.num_seqs = num_seqs;
    a.pool_size = pool_size;
    a.silu = silu != 0;
    a.polls = g_prefill_wait_polls.load(std::memory_order_relaxed);
    const cudaError_t e = gdn::launch_conv(a, taps, dtype == GDN_F16, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    return launched(fn);
}

// What the two forms of the scan ask of their arguments; fills `a`.
static gdn_status ssm_check(const char* fn, gdn::SsmArgs* a, const void* x, const void* dt, const void* B, const void* C, const void* z,
                            const int64_t* strides, const float* A_log, const float* D, const float* dt_bias, float* state_pool,
                            int pool_size, const int64_t* cache_indices, int num_seqs, int64_t T, int H, int P, int G, int N, void* out,
                            int32_t* dev_status) {
    REQUIRE(x && dt && B && C && A_log && dt_bias && state_pool && cache_indices && out && dev_status && strides, GDN_ERR_INVALID_ARG,
            "%s: null pointer", fn);
    const long long inner = static_cast<long long>(H) * P, gn = static_cast<long long>(G) * N;
    const long long least[5] = {inner, H, gn, gn, z ? inner : 0};
    for (int i = 0; i < 5; ++i)
        REQUIRE((i == 4 && !z) || (strides[i] >= least[i] && strides[i] < (1LL << 31) && (i == 1 || strides[i] % 8 == 0)), GDN_ERR_INVALID_ARG,
                "%s: token strides must cover a token, be below 2^31 and (but for dt's) be multiples of 8", fn);
    REQUIRE(aligned(x, 16) && aligned(B, 16) && aligned(C, 16) && aligned(z, 16) && aligned(out, 16) && aligned(state_pool, 16) &&
                aligned(dt, 2) && aligned(A_log, 4) && aligned(D, 4) && aligned(dt_bias, 4) && aligned(cache_indices, 8) && aligned(dev_status, 4),
            GDN_ERR_INVALID_ARG, "%s: x, B, C, z, out and state_pool must be 16-byte aligned", fn);
    REQUIRE(T < (1LL << 31) && static_cast<long long>(num_seqs) * H * (P / 32) < (1LL << 31) && inner < (1LL << 31) && gn < (1LL << 31),
            GDN_ERR_UNSUPPORTED, "%s: T and num_seqs * H * P / 32 must be below 2^31", fn);
    const size_t ob = static_cast<size_t>(T) * inner * 2, sb = static_cast<size_t>(pool_size) * inner * N * 4;
    auto span = [&](int i) { return (static_cast<size_t>(T - 1) * strides[i] + least[i]) * 2; };
    const void* const in[5] = {x, dt, B, C, z};
    for (int i = 0; i < 5; ++i) {
        const size_t b = in[i] ? span(i) : 0;
        REQUIRE(!any_overlap(out, ob, in[i], b) && !any_overlap(state_pool, sb, in[i], b), GDN_ERR_INVALID_ARG,
                "%s: out or state_pool overlaps an input", fn);
    }
    const size_t hb = static_cast<size_t>(H) * 4;
    REQUIRE(!any_overlap(out, ob, state_pool, sb) && !any_overlap(out, ob, A_log, hb) && !any_overlap(out, ob, dt_bias, hb) &&
                !any_overlap(out, ob, D, D ? hb : 0) && !any_overlap(state_pool, sb, A_log, hb) && !any_overlap(state_pool, sb, dt_bias, hb) &&
                !any_overlap(state_pool, sb, D, D ? hb : 0),
            GDN_ERR_INVALID_ARG, "%s: out or state_pool overlaps another buffer", fn);
    std::memset(a, 0, sizeof(*a));
    a->x = static_cast<const uint16_t*>(x);
    a->dt = static_cast<const uint16_t*>(dt);
    a->B = static_cast<const uint16_t*>(B);
    a->C = static_cast<const uint16_t*>(C);
    a->z = static_cast<const uint16_t*>(z);
    a->x_stride = strides[0];
    a->dt_stride = strides[1];
    a->b_stride = strides[2];
    a->c_stride = strides[3];
    a->z_stride = strides[4];
    a->A_log = A_log;
    a->D = D;
    a->dt_bias = dt_bias;
    a->state = state_pool;
    a->slots = cache_indices;
    a->out = static_cast<uint16_t*>(out);
    a->status = dev_status;
    a->T = T;
    a->num_seqs = num_seqs;
    a->pool_size = pool_size;
    a->H = H;
    a->P = P;
    a->G = G;
    return GDN_OK;
}

static gdn_status ssm_sizes(const char* fn, int num_seqs, int64_t T, int pool_size, int H, int P, int G, int N) {
    REQUIRE(num_seqs >= 0 && T >= 0 && pool_size >= 0 && H >= 1 && G >= 1, GDN_ERR_INVALID_ARG,
            "%s: sizes must be num_seqs, T, pool_size >= 0 and H, G >= 1", fn);
    REQUIRE(H % G == 0, GDN_ERR_INVALID_ARG, "%s: H (%d) must be a multiple of G (%d)", fn, H, G);
    REQUIRE((P == 64 || P == 128) && (N == 64 || N == 128), GDN_ERR_UNSUPPORTED, "%s: P and N must be 64 or 128 (got %d and %d)", fn, P, N);
    return GDN_OK;
}

extern "C" gdn_status ssm_decode_step(const void* x, const void* dt, const void* B, const void* C, const void* z,
                                      const int64_t* token_strides, const float* A_log, const float* D, const float* dt_bias,
                                      float* state_pool, int pool_size, const int64_t* cache_indices, int num_seqs, int H, int P,
                                      int G, int N, void* out, int32_t* dev_status, gdn_stream_t stream) {
    const char* fn = "ssm_decode_step";
    gdn_status s = ssm_sizes(fn, num_seqs, num_seqs, pool_size, H, P, G, N);
    if (s != GDN_OK || num_seqs == 0) return s;
    gdn::SsmArgs a;
    s = ssm_check(fn, &a, x, dt, B, C, z, token_strides, A_log, D, dt_bias, state_pool, pool_size, cache_indices, num_seqs, num_seqs, H, P,
                  G, N, out, dev_status);
    if (s != GDN_OK) return s;
    gdn::launch_ssm_steps(a, N, static_cast<cudaStream_t>(stream));
    return launched(fn);
}

extern "C" size_t ssm_prefill_workspace_size(int num_seqs, int64_t T, int H, int P, int N) {
    if (num_seqs < 0 || T < 0 || H < 1 || (P != 64 && P != 128) || (N != 64 && N != 128)) return 0;
    return gdn::ssm_workspace_bytes(num_seqs, T, H, P, N);
}

extern "C" gdn_status ssm_prefill_chunked(const void* x, const void* dt, const void* B, const void* C, const void* z,
                                          const int64_t* token_strides, const float* A_log, const float* D, const float* dt_bias,
                                          float* state_pool, int pool_size, const int64_t* cache_indices, const int64_t* cu_seqlens,
                                          int num_seqs, int64_t T, int64_t max_len, int H, int P, int G, int N, void* out,
                                          void* workspace, size_t workspace_bytes, int32_t* dev_status, gdn_stream_t stream) {
    const char* fn = "ssm_prefill_chunked";
    gdn_status s = ssm_sizes(fn, num_seqs, T, pool_size, H, P, G, N);
    if (s != GDN_OK || num_seqs == 0 || T == 0) return s;
    REQUIRE(max_len >= 0, GDN_ERR_INVALID_ARG, "%s: max_len must not be negative", fn);
    gdn::SsmArgs a;
    s = ssm_check(fn, &a, x, dt, B, C, z, token_strides, A_log, D, dt_bias, state_pool, pool_size, cache_indices, num_seqs, T, H, P, G, N,
                  out, dev_status);
    if (s != GDN_OK) return s;
    REQUIRE(cu_seqlens && aligned(cu_seqlens, 8), GDN_ERR_INVALID_ARG, "%s: null or misaligned cu_seqlens", fn);
    const size_t need = gdn::ssm_workspace_bytes(num_seqs, T, H, P, N);
    REQUIRE(need == 0 || (workspace && workspace_bytes >= need), GDN_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed (got %zu)", fn, need,
            workspace ? workspace_bytes : size_t(0));
    REQUIRE(max_len <= gdn::kSsmSteps || (aligned(workspace, 32) && aligned(state_pool, 32)), GDN_ERR_INVALID_ARG,
            "%s: workspace and state_pool must be 32-byte aligned where max_len is over %d", fn, gdn::kSsmSteps);
    const size_t inner = static_cast<size_t>(H) * P, sb = static_cast<size_t>(pool_size) * inner * N * 4;
    REQUIRE(!any_overlap(workspace, need, out, static_cast<size_t>(T) * inner * 2) && !any_overlap(workspace, need, state_pool, sb),
            GDN_ERR_INVALID_ARG, "%s: workspace overlaps another buffer", fn);
    const size_t gn = static_cast<size_t>(G) * N * 2, hb = static_cast<size_t>(H) * 4;
    const void* const in[5] = {x, dt, B, C, z};
    const size_t least[5] = {inner * 2, static_cast<size_t>(H) * 2, gn, gn, inner * 2};
    for (int i = 0; i < 5; ++i)
        REQUIRE(!in[i] || !any_overlap(workspace, need, in[i], static_cast<size_t>(T - 1) * token_strides[i] * 2 + least[i]), GDN_ERR_INVALID_ARG,
                "%s: workspace overlaps an input", fn);
    REQUIRE(!any_overlap(workspace, need, A_log, hb) && !any_overlap(workspace, need, dt_bias, hb) && !any_overlap(workspace, need, D, D ? hb : 0) &&
                !any_overlap(workspace, need, cu_seqlens, (static_cast<size_t>(num_seqs) + 1) * 8) &&
                !any_overlap(workspace, need, cache_indices, static_cast<size_t>(num_seqs) * 8) && !any_overlap(workspace, need, dev_status, 4),
            GDN_ERR_INVALID_ARG, "%s: workspace overlaps another buffer", fn);
    a.cu = cu_seqlens;
    a.polls = g_prefill_wait_polls.load(std::memory_order_relaxed);
    const cudaError_t e = gdn::launch_ssm_prefill(a, N, max_len, workspace, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    return launched(fn);
}

extern "C" gdn_status add_rms_norm(const void* x, int64_t x_stride, void* residual, gdn_dtype dtype, const float* weight, float eps,
                                   int64_t T, int C, void* out, gdn_dtype out_dtype, float* scale, int group, gdn_stream_t stream) {
    const char* fn = "add_rms_norm";
    REQUIRE(T >= 0 && C >= 1, GDN_ERR_INVALID_ARG, "%s: sizes must be T >= 0 and C >= 1", fn);
    REQUIRE(dtype == GDN_BF16 || dtype == GDN_F16, GDN_ERR_INVALID_ARG, "%s: dtype must be GDN_BF16 or GDN_F16", fn);
    REQUIRE(out_dtype == dtype || out_dtype == GDN_E4M3, GDN_ERR_INVALID_ARG, "%s: out_dtype must be dtype or GDN_E4M3", fn);
    REQUIRE(C % 8 == 0 && C <= 32768, GDN_ERR_UNSUPPORTED, "%s: C must be a multiple of 8, at most 32768 (got %d)", fn, C);
    const bool f8 = out_dtype == GDN_E4M3;
    REQUIRE(f8 == (scale != nullptr) || T == 0, GDN_ERR_INVALID_ARG, "%s: scale is for an 8-bit output, which needs it", fn);
    REQUIRE(group == 0 || (f8 && (group == 32 || group == 64 || group == 128 || group == 256) && C % group == 0), GDN_ERR_UNSUPPORTED,
            "%s: group must be 0, or (8 bits) 32, 64, 128 or 256 and a divisor of C (got %d)", fn, group);
    REQUIRE(T < (1LL << 31), GDN_ERR_UNSUPPORTED, "%s: T must be below 2^31", fn);
    if (T == 0) return GDN_OK;
    REQUIRE(x && weight && out, GDN_ERR_INVALID_ARG, "%s: null pointer", fn);
    REQUIRE(x_stride >= C && x_stride % 8 == 0 && x_stride < (1LL << 31), GDN_ERR_INVALID_ARG,
            "%s: x_stride must be a multiple of 8, at least C and below 2^31", fn);
    REQUIRE(aligned(x, 16) && aligned(residual, 16) && aligned(weight, 16) && aligned(out, 16) && aligned(scale, 4), GDN_ERR_INVALID_ARG,
            "%s: x, residual, weight and out must be 16-byte aligned", fn);
    const size_t xb = (static_cast<size_t>(T - 1) * x_stride + C) * 2, rb = residual ? static_cast<size_t>(T) * C * 2 : 0;
    const size_t ob = static_cast<size_t>(T) * C * (f8 ? 1 : 2), sb = f8 ? static_cast<size_t>(T) * (group ? C / group : 1) * 4 : 0;
    const size_t wb = static_cast<size_t>(C) * 4;
    REQUIRE((out == x && !f8 && x_stride == C) || !any_overlap(out, ob, x, xb), GDN_ERR_INVALID_ARG,
            "%s: out overlaps x (it may be x itself, in 16 bits and dense)", fn);
    REQUIRE(!any_overlap(residual, rb, x, xb) && !any_overlap(out, ob, residual, rb) && !any_overlap(out, ob, weight, wb) &&
                !any_overlap(residual, rb, weight, wb) && !any_overlap(scale, sb, x, xb) && !any_overlap(scale, sb, residual, rb) &&
                !any_overlap(scale, sb, out, ob) && !any_overlap(scale, sb, weight, wb),
            GDN_ERR_INVALID_ARG, "%s: residual, out or scale overlaps another buffer", fn);
    gdn::NormArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.x_stride = x_stride;
    a.residual = static_cast<uint16_t*>(residual);
    a.w = weight;
    a.out = out;
    a.scale = scale;
    a.T = T;
    a.C = C;
    a.lanes = group / 8;
    a.eps = eps;
    gdn::launch_norm(a, dtype == GDN_F16, f8, static_cast<cudaStream_t>(stream));
    return launched(fn);
}
