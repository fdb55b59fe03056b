/*
 * fkl_cache.h - C ABI of the teacher cache in few bits: the top-K ids and logits of
 * fkl_teacher_topk, 8 bytes a slot, packed as they are written and unpacked as the loss reads
 * them.
 *
 * Offline distillation writes the cache once and reads it in every epoch, from storage and over
 * the bus, so its size is what it costs.  A row of K slots becomes a record of 32-bit words in
 * three parts:
 *
 *     scales  2 G words, G = ceil(K / 32): for each 32 slots the largest logit `top` and the step
 *             (float)
 *     codes   ceil(K * bits / 32) words: slot k's code in bits [k bits, (k + 1) bits)
 *     ids     ceil(K * id_bits / 32) words: slot k's id in the same way, id_bits the least number
 *             with V < 2^id_bits
 *
 * (little-endian bit order within the words of a part; unused bits are 0).  Of 32 slots with
 * largest and smallest logit top and low, levels = 2^bits - 2 and step = (top - low) / levels in
 * float,
 *
 *     code = round((top - z) levels / (top - low))  (nearest level, a tie to the even one; 0 where top = low)
 *     z'   = top - code * step                      (each operation rounded to float)
 *
 * so a logit is off by half a step at most, and the largest of each 32 slots by nothing.  The last code,
 * 2^bits - 1, stands for -inf.  A slot that lies more than 4096 below its row's largest logit is stored as -inf: it has
 * no probability in float at any temperature up to 39, and a logit of the type's lowest value would
 * take the resolution of all others.  Slots may have any order; a teacher's, sorted by logit, has the
 * finest steps.  An id outside [0, V) is stored as the id 2^id_bits - 1 and read as -1.  A row that holds a NaN or +inf
 * is read as NaN in all its slots (`top` is NaN).  At K = 100 and V = 201088 a record has 360 bytes in 8 bits
 * and 312 in 4, for the 800 of ids and logits.
 *
 * Conventions (device pointers, streams, errors, ownership) are those of fkl.h.
 */
#ifndef FKL_CACHE_H_
#define FKL_CACHE_H_

#include <stddef.h>
#include <stdint.h>

#include "fkl.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 32-bit words of a row's record; 0 for arguments out of range (1 <= K <= 1024, 1 <= V <= 2^30, bits 4 or 8). */
int32_t fkl_cache_words(int64_t K, int64_t V, int32_t bits);

/*
 * Packs T rows: ids int32 [T][K] and logits float [T][K] into records [T][fkl_cache_words].  4-byte aligned,
 * contiguous; 0 <= T < 2^31.
 */
fkl_status fkl_cache_pack(const int32_t* topk_idx, const float* topk_logits, int64_t T, int64_t K, int64_t V,
                          int32_t bits, uint32_t* records, void* stream);

/* Unpacks T records into ids int32 [T][K] and logits float [T][K]. */
fkl_status fkl_cache_unpack(const uint32_t* records, int64_t T, int64_t K, int64_t V, int32_t bits,
                            int32_t* topk_idx, float* topk_logits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FKL_CACHE_H_ */
