// Host side shared by the calls on the paged 8-bit cache.
#pragma once
#include "kv8_common.cuh"

namespace qg {

// What every such call is given.
struct Kv8Args {
    int8_t *kq, *vq;
    float *ks, *vs;
    const int32_t *table, *starts, *lengths;
    int64_t B, rows, pages, page, heads, D, table_cols;
};
int check_kv8(const Kv8Args& a);
int check_kv8_rows(int dtype, const void* X, int64_t ld, int64_t values, int64_t rows);
void kv8_params(const Kv8Args& a, Kv8Cache* c, Kv8Batch* bt);

}  // namespace qg
