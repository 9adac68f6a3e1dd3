// serve_internal.h -- internal declarations of the drafted-token verification
// operators: the group-scaled 4-bit product (k_q4_group.hip), the cache plan
// and append (k_kv.hip) and the attention over it (tree_attention.h).
#pragma once

#include "qmm_internal.h"

namespace qmm {

// ------------------------------------------------------------------------
// Device layout of a group-scaled 4-bit weight.  Codes are records of 128 k
// x 16 columns, strip-major like q4_1's:
//   record (strip, q) at (strip*NQ + q) * 1024; 16-byte chunk `lane` holds,
//   for column lane%16 and k-octet g = lane/16, a 4-byte word per block
//   i = 0..3 with the codes of k = 128q + 32i + 8g + e: element e in nibble
//   e/2 (e even) or 4 + e/2 (e odd), so that elements 2p and 2p+1 come out of
//   one shift and one mask as the low and high half of a register.
// Behind the codes, one 4-byte word per group: the scale as fp32 with the
// zero in its low four bits (an fp16 or bf16 scale leaves at least 13 zero
// bits there).  Word w of a record's GPR = max(128/group, 1) and column c:
//   group <  128: ((strip*NQ + q)*16 + c)*GPR + w
//   group >= 128: (strip*NG + q*128/group)*16 + c,  NG = ceil(K/group)
// Padding has code 0 and word 0.
// ------------------------------------------------------------------------
constexpr int kQ4gRecBytes = 1024;

struct Q4gLayout {
    int64_t K, N, NQ, NS, NG, gpr, words_off, total;
};

inline Q4gLayout q4g_layout(int64_t K, int64_t N, int64_t group) {
    Q4gLayout L;
    L.K = K;
    L.N = N;
    L.NQ = ceil_div(K, 128);
    L.NS = ceil_div(N, 16);
    L.NG = ceil_div(K, group);
    L.gpr = group < 128 ? 128 / group : 1;
    L.words_off = L.NS * L.NQ * kQ4gRecBytes;
    L.total = L.words_off + 64 * (group < 128 ? L.NS * L.NQ * L.gpr : L.NS * L.NG);
    return L;
}

// Threads of a grid, less than 2^32, in whole workgroups of up to 512.  The repack
// takes 64 for a record, the product of few rows 512 for a strip.
constexpr int64_t kGridThreads = ((int64_t)1 << 32) - 512;
inline bool q4g_fits(const Q4gLayout &L) { return L.NS <= kGridThreads / 512 && L.NS * L.NQ <= kGridThreads / 64; }

struct Q4gParams {
    const uint8_t *recs;    // code records
    const uint32_t *words;  // group words
    const void *X;
    void *Y;
    int64_t ldx, ldy;
    int M, K, N, NQ, NS, NG;
    int rpg;                // records per group (group >= 128), else 1
    int gpr;                // groups per record (group < 128), else 1
    int x_vec;              // rows of X are 16-byte aligned
    void *xa;               // laid-out activations, their group sums (16-bit rows), partial products (workspace)
    float *xs, *part;
};

// How a product is cut.  laid: the activations are laid out first (more than 16
// rows, or rows that 16-byte loads cannot read); mt: 16-row tiles of a wavefront;
// parts: record ranges of the workgroups of one tile of columns.
constexpr int kQ4gRowsLds = 29 * 1024;  // rows of up to 16 that are copied to LDS: four workgroups to a CU
constexpr int64_t kQ4gMaxRows = 16 * 65520;  // one grid covers the 16-row tiles

struct Q4gShape {
    bool laid;
    int mt, tiles, parts;
    int64_t xs_off, part_off, total;
};

inline Q4gShape q4g_shape(int64_t M, int64_t N, int64_t terms, bool vec, const Q4gLayout &L) {
    Q4gShape z{};
    z.laid = M > 16 || !vec || terms == 3;
    if (!z.laid) return z;
    // four tiles: 27.0 us against 29.7 for 14336 x 4096, M = 64; three terms of them do not fit LDS
    z.mt = M > 32 && terms == 1 ? 4 : M > 16 ? 2 : 1;
    z.tiles = (int)round_up(ceil_div(M, 16), z.mt);
    // as many workgroups as are resident and no more (they would wait for a second
    // turn), where the records allow 4 to each: two to a CU for up to 16 rows, whose
    // partial sums are small (4100 x 11003, M = 5 fp32: 19.4 us a call against
    // 22.6), one for more (14336 x 4096, M = 32, 64: 21.3, 27.0 against 25.2, 30.5)
    const int64_t blocks = ceil_div(L.NS, 8) * (z.tiles / z.mt);
    int64_t parts = (M > 16 ? 256 : 512) / blocks;
    if (parts > L.NQ / 4) parts = L.NQ / 4;
    z.parts = parts > 1 ? (int)parts : 1;
    z.xs_off = round_up(z.tiles * L.NQ * 4 * terms * 1024, 256);
    // sums of 16-bit rows only; they are copied 1 KiB at a time
    z.part_off = z.xs_off + (terms == 3 ? 0 : round_up(z.tiles * L.NQ * L.gpr * 64 + 1024, 256));
    z.total = z.part_off + (z.parts > 1 ? z.parts * M * N * 4 : 0);
    return z;
}

hipError_t launch_q4g_repack(const uint8_t *codes, int64_t ldc, const void *scales, bool bf16, int64_t lds,
                             const uint8_t *zeros, int64_t ldz, int64_t group, const Q4gLayout &L,
                             uint8_t *packed, hipStream_t s);
hipError_t launch_q4g_matmul(const Q4gParams &p, qmm_dtype xt, int gpr, const Q4gShape &z, hipStream_t s,
                             const char **variant);

struct KvPlanParams {
    const int32_t *ctx_lens, *new_lens;
    int32_t *table;
    int64_t ld_table;
    const int32_t *free_pages, *free_begin;
    int32_t *cu_new, *positions, *info;
    int64_t *slots;
    int R, width, page, n_free, max_tokens;
};

constexpr int kPlanMaxRequests = 8192;  // cu_new and first pages sit in LDS
hipError_t launch_kv_plan(const KvPlanParams &p, hipStream_t s);

struct KvAppendParams {
    const void *src[2];      // K, V
    int64_t tok[2], head[2]; // their strides
    void *dst[2];
    float *scale[2];
    const int64_t *slots;
    int64_t n_slots;
    int64_t page_stride, token_stride, head_stride;
    int64_t sp_stride, st_stride, sh_stride;
    int64_t rows;            // T * H
    int H, D, page;
};

// log2 of the lanes of a row: 8 values each.
inline int kv_append_lanes_log2(int64_t D) {
    int l = 0;
    while ((8 << l) < D) ++l;
    return l;
}

// vec: the rows of K and V allow aligned 16-byte accesses.
hipError_t launch_kv_append(const KvAppendParams &p, qmm_dtype xt, qmm_dtype ct, bool vec, hipStream_t s);
// The other way: src are the rows that are written, dst the cache that is read.
hipError_t launch_kv_gather(const KvAppendParams &p, qmm_dtype xt, qmm_dtype ct, bool vec, hipStream_t s);

// What a workgroup of the tree attention leaves for the second launch: the
// shared item whose last part is its own (rows 0: none), whether a sum of its was
// not finite, and its run: request r, whose units begin at base, units u .. u1-1.
struct TreeHeader {
    int rows, first_wg, hk, row0, first, bad, r;
    int64_t base, u, u1;
};

struct TreeParams {
    const void *Q;
    void *O;
    int64_t q_tok, q_head, o_tok, o_head;
    const void *k, *v;
    const float *k_scale, *v_scale;
    int64_t page_stride, token_stride, head_stride, sp_stride, st_stride, sh_stride;
    const int32_t *table, *ctx_lens, *cu_new;
    int64_t ld_table;
    const uint8_t *mask;
    int64_t ld_mask;
    int T, Hq, Hkv, G, D, R, width, page, num_pages, mask_cols;
    int window, sinks;       // window attention
    uint32_t page_mul;       // j / page = j * page_mul >> page_shift for j < 2^31
    int page_shift;
    float scale;             // its size, times log2(e)
    int q_flip;              // sign bits to flip in a pair of Q's elements: a negative scale
    int q_vec, o_vec;        // aligned 16-byte loads of Q, 8-byte stores of O
    TreeHeader *hdr;         // per workgroup
    float *part;             // two slots per workgroup, slot_rows x (m, l, dk sums)
    int slot_rows, wgs;
};

constexpr int kTreeWorkgroups = 512;  // two per CU are resident
constexpr int kTreeItem = 3;          // what an item costs beside its key blocks, in blocks
// Keys of a request.  The kernels count keys in 32 bits, 64 at a time: the step
// past the last key must not wrap, or a loop over the keys would not end.
constexpr int64_t kTreeMaxKeys = INT32_MAX - 63;
constexpr int tree_keys(int dk) { return dk <= 128 ? 64 : 32; }  // a step's

// How a call is cut: dk, the head dimension the kernel works on; 16-row tiles
// of a wavefront (four to a workgroup); workgroups; workspace.
struct TreeShape {
    bool few;  // 4-bit rows, and few rows a request: k_few4
    int dk, mt, heads, slot_rows;
    int64_t wgs;
    int64_t hdr_bytes, total;
};

// Few rows over 4-bit rows: the wavefronts of a workgroup take a cache head each where heads
// come in eights or fours, else a quarter of a block's keys each.  A head each means
// that a share leaves sums of all their rows, so it is taken where a share has half as
// many blocks of 32 keys as a head has rows, and two at least.  us a call with and
// without, tokens x (query over cache heads):
//   1 x 131000 keys, 1 x (32 / 8)     50 / 71       4 x 2000, 9 x (16 / 8)     29 / 19
//   16 x 4096, 4 x (32 / 8)           35 / 40       1 x 1000, 1 x (16 / 8)     18 / 15
//   61 x 16448, 1 x (32 / 8)         233 / 370      64 x 1000, 1 x (32 / 8)    30 / 31
constexpr int few_workgroups(int mt, int heads) { return heads == 8 ? 256 : mt == 1 && heads == 4 ? 768 : 512; }
inline int few_heads(int64_t Hkv, int64_t R, int64_t keys, int64_t rows, int mt) {
    const int64_t least = rows > 4 ? ceil_div(rows, 2) : 2;
    for (int heads : {8, 4})
        if (Hkv % heads == 0 && Hkv / heads * ceil_div(keys, 32) >= ceil_div(least * few_workgroups(mt, heads), R)) return heads;
    return 1;
}
constexpr int few_waves(int heads) { return heads == 8 ? 8 : 4; }
constexpr int few_keys(int heads) { return heads == 1 ? 128 : 32; }
constexpr int few_item(int heads) { return heads == 1 ? 2 : 6; }

inline TreeShape tree_shape(int64_t T, int64_t G, int64_t R, int64_t Hkv, int64_t D, int64_t keys, bool q4) {
    TreeShape z{};
    z.dk = D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : 256;
    // two tiles of a wavefront where requests have more than one 64-row tile on
    // average.  us a call with two against one, by cache type (ragged batches of
    // 8 cache heads of 128, rows a request on average):
    //   requests x keys, rows     bf16          fp16          int8
    //   16 x 8192, 48             85 / 81       85 / 82       80 / 69
    //   16 x 8192, 69             93 / 102      93 / 101      89 / 93
    //   16 x 8192, 118            115 / 143     117 / 143     126 / 135
    //   1 x 131000, 128           143 / 176     147 / 182     152 / 187
    //   32 x 32768, 97            623 / 971     639 / 997     659 / 874
    //   4 x 2048, 192             37 / 33       37 / 33       39 / 33
    // The lengths lie on the device, so the last line's loss is not told from the
    // others' gain.  The int8 form of two tiles does not fit its registers (12 are
    // spilled) and gains all the same.
    z.mt = z.dk <= 128 && T * G > 64 * R ? 2 : 1;
    z.few = q4 && T * G <= (z.dk <= 128 ? 32 : 16) * R;
    if (z.few) z.mt = T * G > 16 * R ? 2 : 1;
    z.heads = z.few ? few_heads(Hkv, R, keys, ceil_div(T * G, R), z.dk > 128 ? 2 : z.mt) : 1;
    const int64_t rows = (z.few ? 16 : 64) * z.mt, kb = z.few ? few_keys(z.heads) : tree_keys(z.dk);
    z.slot_rows = (int)(z.heads * (T * G < rows ? T * G : rows));
    // fewer workgroups where there cannot be as many key blocks
    const int64_t tiles = ceil_div(T * G, rows) + (R < T ? R : T), groups = Hkv / z.heads;
    const int64_t blocks = (keys > kb ? ceil_div(keys, kb) : 1) + (z.few ? few_item(z.heads) : kTreeItem);
    z.wgs = z.few ? few_workgroups(z.dk > 128 ? 2 : z.mt, z.heads) : kTreeWorkgroups;
    if (tiles < z.wgs && groups < z.wgs && blocks < z.wgs && tiles * groups * blocks < z.wgs) z.wgs = tiles * groups * blocks;
    z.hdr_bytes = round_up(z.wgs * (int64_t)sizeof(TreeHeader), 256);
    z.total = z.hdr_bytes + z.wgs * 2 * z.slot_rows * (z.dk + 2) * 4;
    return z;
}

hipError_t launch_tree_attention(const TreeParams &p, const TreeShape &z, qmm_dtype ct, hipStream_t s,
                                 const char **variant);
hipError_t launch_tree_attention_q4(const TreeParams &p, const TreeShape &z, hipStream_t s);
hipError_t launch_window_attention(const TreeParams &p, const TreeShape &z, qmm_dtype ct, hipStream_t s,
                                   const char **variant);
hipError_t launch_window_attention_q4(const TreeParams &p, const TreeShape &z, hipStream_t s);

}  // namespace qmm
