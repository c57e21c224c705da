// What attention to shared prefixes (kda_attn_prefix.cu) leaves beside the parts of the rest of each row
// (kda_attn_stream.cuh), for the join of both.
#pragma once

#include <stdint.h>

#include "kda_internal.cuh"

namespace kda {

constexpr int kPrefixTile = 128;               // tokens, and query rows, of a tile
constexpr int kPrefixSlots = 2 * kPrefixTile;  // query rows that a CTA works on
constexpr int32_t kTailHome = -1, kTailNone = -2;

// Where the parts of a query row's prefix are: the first is in the row's home, each further CTA of its item has
// one in its own slots. per: parts of each CTA (two where its two groups of warps share the row's tokens).
struct alignas(16) PrefixCut {
    int32_t per, slot, cta, ctas;  // cta, ctas: the CTAs behind the first
};

struct PrefixParts {
    int32_t *start;   // [batch]: the row's tokens before this one are in the parts (0: none)
    PrefixCut *cuts;  // [batch][query heads]
    int32_t *tails;   // [batch][query heads]: where the rest of the row is: a share of the token stream whose Cut says
                      // so, kTailHome or kTailNone
    float2 *ml;       // [parts]: maximum (log2 units), sum of 2^(x - maximum)
    float *o;         // [parts][128]
    int32_t heads;    // batch * query heads; parts: a home of two for each and one of the rest, then kPrefixSlots
                      // for each CTA
    int32_t ctas;

    // Parts of a row's prefix; none where the record makes no sense (a CTA that gave up wrote none).
    __device__ __forceinline__ int parts_of(const PrefixCut &c) const {
        const bool sane = (c.per == 1 || c.per == 2) && c.slot >= 0 && c.slot < kPrefixSlots / c.per && c.cta >= 0 && c.ctas >= 0 &&
                          c.cta <= ctas && c.ctas <= ctas - c.cta;
        return sane ? c.per * (1 + c.ctas) : 0;
    }
    __device__ __forceinline__ int64_t part_at(const PrefixCut &c, int64_t head, int i) const {
        if (i < c.per) return (int64_t)i * heads + head;
        const int j = i - c.per, behind = c.per == 2 ? j >> 1 : j, w = c.per == 2 ? j & 1 : 0;
        return 3 * (int64_t)heads + (int64_t)(c.cta + behind) * kPrefixSlots + w * kPrefixTile + c.slot;
    }
};

__host__ __device__ __forceinline__ int64_t prefix_layout(PrefixParts *x, char *base, int64_t batch, int64_t q_heads, int64_t ctas) {
    const int64_t heads = batch * q_heads, parts = 3 * heads + ctas * kPrefixSlots;
    int64_t n = 0;
    if (x) x->start = reinterpret_cast<int32_t *>(base + n);
    n += (batch * 4 + 15) / 16 * 16;
    if (x) x->cuts = reinterpret_cast<PrefixCut *>(base + n);
    n += heads * (int64_t)sizeof(PrefixCut);
    if (x) x->tails = reinterpret_cast<int32_t *>(base + n);
    n += (heads * 4 + 15) / 16 * 16;
    if (x) x->ml = reinterpret_cast<float2 *>(base + n);
    n += (parts * 8 + 15) / 16 * 16;
    if (x) x->o = reinterpret_cast<float *>(base + n);
    n += parts * kHeadDim * 4;
    if (x) x->heads = (int32_t)heads, x->ctas = (int32_t)ctas;
    return n;
}

struct AttnPrefixArgs {
    AttnDecodeArgs d;
    const int32_t *cu_groups, *prefix_lens;
    int32_t groups;
    PrefixParts x;
};

int64_t attn_prefix_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int64_t capacity, int32_t sms);
cudaError_t launch_attn_prefix(const AttnPrefixArgs &a, cudaStream_t stream);

}  // namespace kda
