// paged_q4.cuh -- the 4-bit KV cache in pages: where the bytes of a token lie, and
// the parameters that the kernels over it share.
//
// A page holds page_size tokens of every kv head: [kv head][page_size / 16] records
// of 16 tokens of one kv head, 18 * head_dim bytes each (nb = head_dim / 32 blocks
// of 32 values, each a Q4_0 block: value = d * (code - 8), d f16):
//   0            K codes   16 rows of head_dim / 2 bytes, one for each token
//   8 head_dim   K scales  f16 [16][nb]
//   9 head_dim   V codes   8 * head_dim bytes, tokens innermost
//  17 head_dim   V scales  f16 [16][nb]
// Byte i < 16 of a block holds value i in its low nibble and value i + 16 in its
// high nibble, as in Q4_0.  The order of the bytes is that in which the lanes of a
// warp need them for m16n8k16 products, lane = 4 g + t:
//   K: 4-byte word t of block b (bytes 4 t .. 4 t + 3) is word t * nb + b of the row,
//      so that a lane's words of one token are one vector load.
//   V: byte p = 16 b + i of token 4 t + j is byte j of word r = p / 8 of lane
//      (g = p % 8, t); a lane's words lie together in runs of kVRun(nb).
// Any order of the values of a sum gives the same sum: the query is laid out in the
// same order as the key's words, and the softmax weights in that of the tokens.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace rz {

__host__ __device__ constexpr int q4_record_bytes(int head_dim) { return 18 * head_dim; }
__host__ __device__ constexpr int q4_v_run(int nb) { return nb % 2 == 0 ? 4 : 2; }

// byte i of block b of token tok (0..15), from the record's start
__host__ __device__ constexpr int q4_k_byte(int nb, int tok, int b, int i)
{
    return tok * 16 * nb + ((i / 4) * nb + b) * 4 + i % 4;
}
__host__ __device__ constexpr int q4_v_byte(int nb, int tok, int b, int i)
{
    const int p = 16 * b + i, r = p / 8, lane = (p % 8) * 4 + tok / 4, run = q4_v_run(nb);
    return 9 * 32 * nb + ((r / run) * 32 + lane) * run * 4 + (r % run) * 4 + tok % 4;
}
__host__ __device__ constexpr int q4_k_scale(int nb, int tok) { return 8 * 32 * nb + tok * nb * 2; }
__host__ __device__ constexpr int q4_v_scale(int nb, int tok) { return 17 * 32 * nb + tok * nb * 2; }

// A 4-bit paged cache (validated by the C-ABI layer): page_size = 16 << page_log.
struct PagedKv {
    uint8_t *pages;
    int64_t n_pages;
    int page_log;  // log2(page_size / 16)
    int n_kv_heads, head_dim;
};

}  // namespace rz
