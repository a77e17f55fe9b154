// Host side of the attention over the paged cache: which kernel takes a call,
// and its workspace.
#include "paged.cuh"

#include <algorithm>
#include <mutex>

namespace sq {
namespace {

__device__ unsigned int g_paged_error;

constexpr int64_t kCounterBytes = 2 * kMaxWorkers * 4;
constexpr int64_t kPieceRows = 128;  // rows of a partial result, the largest kernel's

// Device address of the error word, looked up on a device's first call.
sq_status error_word(int device, unsigned **out) {
    static std::mutex mu;
    static unsigned *known[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    unsigned *&p = known[device & 63];
    if (!p) {
        void *v = nullptr;
        if (cudaGetSymbolAddress(&v, g_paged_error) != cudaSuccess || !v) {
            (void)cudaGetLastError();
            return SQ_ERR_CUDA;
        }
        p = static_cast<unsigned *>(v);
    }
    *out = p;
    return SQ_OK;
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Whether a sequence's rows (tokens x heads of a key/value head's group) go to the
// kernel for few rows: one tile of at most 16 of its rows, whose cost is the cache's
// way through the SMs.  The other kernel's tile of 128 rows costs the same for 8
// rows as for 128.  Measured at 16 rows, few against many (32 / 8 heads of 128, 4
// tokens a sequence; us): 1 sequence of 300 keys 21 and 27, 16 of 4000 84 and 98
// (bf16), 80 and 80 (fp16), 64 of 4000 203 and 307, 184 and 234, heads of 64 129
// and 248, 119 and 191.  Two tiles of few rows read and multiply everything twice:
// 406 against 307 us.
bool few_rows(int64_t tokens, int G) { return std::max<int64_t>(1, tokens) * G <= 16; }

// Whether the shared prefix is read in front of every item's own keys instead of
// once for all rows, in a launch of its own.  What the launch costs by itself is
// the start and the end of its items, the prefix's state written and read back,
// and the wait for it; what it saves is the prefix's key tiles for the row tiles
// that it has fewer of, one for every sequence at most.  Measured (heads 32 / 8
// of 128, bf16, own keys up to 512, one token a sequence; separate against in
// front): 16 sequences behind 1000 positions 57 and 27 us, 64: 66 and 53; 64
// behind 3000: 74 and 115, 16 behind 8000: 90 and 82.  The times meet at 40 to 50
// key tiles of 128 per SM, and at 20 to 27 with many rows (fp16, 5 to 8 tokens,
// 24 sequences behind 1000: 88 and 72 us, behind 3000: 92 and 102).  Where the
// sequences fill two row tiles each and more, the prefix in front costs less than
// its state's way through memory whatever its length (bf16, 64 sequences of 1 to
// 257 tokens behind 1000 positions: 944 and 782 us, behind 8000: 2838 and 2792).
// tokens: what T, B and max_q leave possible (a padded batch has fewer than T).
bool prefix_in_front(const PagedArgs &a, int64_t max_q, int64_t tokens, int sms) {
    const bool few = few_rows(max_q, a.G);
    if (!few && tokens * a.G >= 256 * (int64_t)a.B) return true;
    const int64_t tiles = (int64_t)std::min(a.B, a.T) * a.Hkv * ((a.prefix_len + 127) / 128);
    return tiles <= (few ? 40 : 20) * (int64_t)sms;
}

}  // namespace

// counters | partial maxima and sums | partial outputs | the prefix's maxima
// and sums | the prefix's outputs
sq_status paged_workspace_bytes(int64_t T, int64_t Hq, int64_t D, int64_t prefix_len,
                                size_t *bytes) {
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    const int64_t rows = 2 * (int64_t)di.sms * kPieceRows;
    int64_t n = kCounterBytes + up256(rows * 8) + up256(rows * D * 4);
    if (prefix_len > 0) n += up256(T * Hq * 8) + up256(T * Hq * D * 4);
    *bytes = (size_t)n;
    return SQ_OK;
}

sq_status launch_paged_attention(const PagedCall &c, cudaStream_t st) {
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    if (di.sms * 8 > kMaxWorkers) return SQ_ERR_UNSUPPORTED;
    PagedArgs a = {};
    if ((rc = error_word(di.device, &a.error)) != SQ_OK) return rc;
    a.Q = c.Q;
    a.O = c.O;
    a.ldq = c.ldq;
    a.block_table = c.block_table;
    a.q_start = c.q_start;
    a.kv_len = c.kv_len;
    a.prefix_pages = c.prefix_pages;
    a.max_pages = c.max_pages;
    char *w = static_cast<char *>(c.workspace);
    const int64_t rows = 2 * (int64_t)di.sms * kPieceRows;
    a.counters = reinterpret_cast<unsigned *>(w);
    w += kCounterBytes;
    a.part_ml = reinterpret_cast<float2 *>(w);
    w += up256(rows * 8);
    a.part_o = reinterpret_cast<float *>(w);
    w += up256(rows * c.D * 4);
    if (c.prefix_len > 0) {
        a.prefix_ml = reinterpret_cast<float2 *>(w);
        w += up256(c.T * c.Hq * 8);
        a.prefix_o = reinterpret_cast<float *>(w);
    }
    a.T = (int)c.T;
    a.B = (int)c.B;
    a.Hq = (int)c.Hq;
    a.Hkv = (int)c.Hkv;
    a.G = (int)(c.Hq / c.Hkv);
    a.g_inv = (65536 + a.G - 1) / a.G;  // n e < 2^16 for the excess e < G of g_inv G over 2^16
    a.num_pages = (int)c.num_pages;
    a.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6
                   : c.page_size == 128 ? 7 : 8;
    a.prefix_len = (int)c.prefix_len;
    a.cap = (int)(c.max_pages * c.page_size);
    // A power of two, so that a logit's product with it is exact: however large a row's
    // maximum is, the largest key's exponent is as formed for the maximum, and its
    // probability what it should be.  The rest is the queries' (one rounding each, 2^-24).
    // Not zero, so that a masked logit's -inf stays -inf under it, and large enough for
    // the factors of fp16 rows; a scale below that is zero: no query counts.
    const float scale = fabsf(c.scale) * 1.4426950408889634f;
    int exponent = 0;
    (void)frexpf(std::max(scale, 0x1p-100f), &exponent);
    exponent = std::min(exponent, 127);
    a.scale = ldexpf(1.0f, exponent);
    a.q_factor = scale < 0x1p-100f ? 0.0f : copysignf(ldexpf(scale, -exponent), c.scale);
    const bool bf16 = c.cache_type == SQ_CACHE_BF16;
    const int64_t max_q = std::min(c.max_q, c.T), tokens = std::min(c.T, max_q * c.B);
    const bool front = c.prefix_len > 0 && prefix_in_front(a, max_q, tokens, di.sms);
    for (int phase = c.prefix_len > 0 && !front ? 1 : 0; phase >= 0; --phase) {
        a.prefix_phase = phase;
        const int64_t most = phase ? tokens : max_q;
        const bool few = few_rows(most, a.G);
        const int r = few ? (std::max<int64_t>(1, most) * a.G <= 8 ? 8 : 16) : 128;
        const int kt = few ? 16 : 128;
        a.after_prefix = few && !phase && c.prefix_len > 0 && !front;
        a.tpt = r / a.G;
        a.kstart = phase ? 0 : a.prefix_len / kt * kt;
        a.front_tiles = front ? (a.prefix_len + kt - 1) / kt : 0;
        a.front_shift = front ? a.front_tiles * kt - a.kstart : 0;
        // the longest line that the sizes allow: every sequence as long as its row
        // of the table, and a row tile of its own begun
        const int64_t tiles = (c.T + a.tpt - 1) / a.tpt + (phase ? 0 : c.B);
        const int64_t keys = ((phase ? 0 : c.max_pages * c.page_size) + c.prefix_len) / kt + 16;
        if (tiles * c.Hkv > ((int64_t)1 << 31) / keys) return SQ_ERR_UNSUPPORTED;
        rc = few ? launch_paged_rows(a, c.k_cache, c.v_cache, (int)c.D, bf16, r, di.sms, st)
                 : launch_paged_tiles(a, c.k_cache, c.v_cache, (int)c.D, bf16, di.sms, st);
        if (rc != SQ_OK) return rc;
    }
    return SQ_OK;
}

sq_status paged_take_error(cudaStream_t st) {
    unsigned int word = 0;
    if (cudaMemcpyFromSymbolAsync(&word, g_paged_error, sizeof(word), 0, cudaMemcpyDeviceToHost,
                                  st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return SQ_ERR_CUDA;
    if (word != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbolAsync(g_paged_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice,
                                    st) != cudaSuccess ||
            cudaStreamSynchronize(st) != cudaSuccess)
            return SQ_ERR_CUDA;
        return SQ_ERR_TIMEOUT;
    }
    return SQ_OK;
}

}  // namespace sq
