/*
 * fsdpshard_embedding.h -- C ABI of libfsdpshard.so, the embedding: where a step's tokens enter the
 * model, and where its gradient leaves it as one more tensor's contribution to the flat vector of
 * fsdpshard.h (bf16 for reduce_shard and adamw_shard_step, or float32 kept over micro-batches).
 *
 *   embedding_lookup   rows of a table for given tokens, scaled
 *   embedding_grad     the table's gradient: rows of equal tokens added up
 *
 * The conventions of fsdpshard.h hold: device pointers owned by the caller, no allocation, no
 * memset, no synchronisation (so every call can be captured in a HIP graph), argument errors found
 * before anything is enqueued, a status returned.  The same call gives the same bits each time:
 * sums have a fixed order, and there are no atomic additions of floating-point values.
 */
#ifndef FSDPSHARD_EMBEDDING_H
#define FSDPSHARD_EMBEDDING_H

#include "fsdpshard_logits.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FSDPSHARD_MAX_DIM ((int64_t)1 << 20)
#define FSDPSHARD_MAX_TOKENS ((int64_t)1 << 24)     /* of one embedding_grad call */

/* A matrix of `rows` rows of `cols` values, `row_stride` elements apart. */
typedef struct fsdpshard_matrix {
    void* data;            /* device, aligned to its element                                  */
    int64_t rows;          /* >= 0                                                            */
    int64_t cols;          /* 1 .. FSDPSHARD_MAX_DIM                                          */
    int64_t row_stride;    /* elements from a row to the next, >= cols (any when rows <= 1)   */
    int32_t dtype;         /* fsdpshard_dtype                                                 */
} fsdpshard_matrix;

/*
 * embedding_lookup -- out[t] = scale * table[ids[t]] for every token t of out->rows.
 * An id below 0 is a position without a token and gives zeros; an id >= table->rows is not read
 * and gives NaN.  One float32 product, one rounding to out's type (scale 1 and equal types: a copy, in
 * which a NaN stays a NaN, not always its bits).
 *
 *   table  [vocab, dim]; vocab up to FSDPSHARD_MAX_VOCAB.  It may be a tensor's place in a flat
 *          vector: any alignment of its element
 *   ids    device, out->rows int64 tokens
 *   out    [tokens, dim], any of the types; tokens up to 2^44.  Elements between rows are not
 *          written.  It may not overlap another buffer of the call
 *   scale  finite
 * Errors: INVALID_ARG (nulls, sizes, scale, overlaps), ALIGNMENT, UNSUPPORTED (dim or vocab too
 *         large), OVERFLOW (extents beyond int64), HIP.
 */
int embedding_lookup(const fsdpshard_matrix* table, const int64_t* ids,
                     const fsdpshard_matrix* out, float scale, void* stream);

/*
 * embedding_grad -- the gradient of the table for the gradient dout of embedding_lookup's out:
 *     d[v] = scale * sum of dout[t] over the tokens t with ids[t] = v
 *   accumulate = 0   dtable[v] = d[v] for every row v (zeros where no token is v)
 *   accumulate = 1   dtable[v] += d[v]; rows without a token are neither read nor written
 * Tokens with an id below 0 or >= dtable->rows take no part, whatever their rows of dout hold.
 * Sums are float32 in the order of the tokens, of at most 64 terms, of which at most tokens / 2^17 + 2 are
 * added up in float32; what a row's tokens have beyond that is joined in float64.  One rounding to
 * dtable's type.
 *
 *   ids        device, dout->rows int64 tokens
 *   dout       [tokens, dim]; tokens up to FSDPSHARD_MAX_TOKENS
 *   dtable     [vocab, dim], any of the types; the same dim.  It may be a tensor's place in a flat
 *              vector: any alignment of its element.  Elements between rows are not written
 *   scale      finite
 *   workspace  device, 16-byte aligned scratch of >= embedding_grad_workspace_bytes(tokens, vocab,
 *              dim) bytes (-1: sizes out of range).  Calls that may overlap need one each
 * No written buffer may overlap another buffer of the call.
 * Errors: as embedding_lookup, and CAPACITY (workspace too small), UNSUPPORTED (too many tokens).
 */
int64_t embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim);
int embedding_grad(const int64_t* ids, const fsdpshard_matrix* dout,
                   const fsdpshard_matrix* dtable, float scale, int32_t accumulate,
                   void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FSDPSHARD_EMBEDDING_H */
