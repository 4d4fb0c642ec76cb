// kda_ssm.cu -- launches the selective state space scan of prompts.
#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

bool multiple(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// Rows of a tensor that can be read n elements of `size` bytes at a time.
bool rows_of(const void* p, int64_t ld, int64_t tokens, int size, int n) {
    return !p || (multiple(p, static_cast<uintptr_t>(size * n)) && (tokens < 2 || ld % n == 0));
}
}  // namespace

void set_ssm_vectors(SsmArgs* a) {
    a->vec = a->dim / a->groups % 4 == 0 && rows_of(a->x, a->ldx, a->tokens, 2, 4) && rows_of(a->z, a->ldz, a->tokens, 2, 4) &&
             rows_of(a->dt, a->lddt, a->tokens, a->dt_f32 ? 4 : 2, 4);
    a->vec8 = a->vec && a->dim / a->groups % 8 == 0 && rows_of(a->x, a->ldx, a->tokens, 2, 8) && rows_of(a->z, a->ldz, a->tokens, 2, 8) &&
              (a->dt_f32 || rows_of(a->dt, a->lddt, a->tokens, 2, 8));
    const int size = a->bc_f32 ? 4 : 2;
    a->vec_bc = a->nstate % 4 == 0 && rows_of(a->B, a->ldb, a->tokens, size, 4) && rows_of(a->C, a->ldc, a->tokens, size, 4);
}

cudaError_t launch_ssm_prefill(SsmArgs a, cudaStream_t stream, int* launches) {
    if (a.N <= 0 || a.dim <= 0) return cudaSuccess;
    set_ssm_vectors(&a);
    const int64_t bc = a.bc_f32 ? 4 : 2;
    a.tile_x = kSsmTile * a.ldx * 2;
    a.tile_z = kSsmTile * a.ldz * 2;
    a.tile_dt = kSsmTile * a.lddt * (a.dt_f32 ? 4 : 2);
    a.tile_b = kSsmTile * a.ldb * bc;
    a.tile_c = kSsmTile * a.ldc * bc;
    a.tile_out = kSsmTile * a.dim;
    if (a.nstate <= 16) return ssm_prefill_16(a, stream, launches);
    if (a.nstate <= 32) return ssm_prefill_32(a, stream, launches);
    return ssm_prefill_64(a, stream, launches);
}

}  // namespace kda
