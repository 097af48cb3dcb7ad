// Host helpers that every C entry point shares: the thread's error message,
// checks of tensor descriptors, the optional index checks.  Defined in
// gdr_api.cpp where nothing else is said.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "gdr.h"

namespace gdr {

// Records the message of a failed call and returns `code`.
int fail(int code, const char* fmt, ...);
void clear_error();

bool present(const gdr_tensor* t);
bool empty(const gdr_tensor* t);
bool missing(const gdr_tensor* t);
bool aligned16(const void* p);
const char* dtype_name(int32_t d);
int64_t vec_mult(int32_t dtype);

int check_tensor(const char* fn, const char* name, const gdr_tensor* t, int ndim,
                 const int64_t* shape, bool allow_f32, bool allow_bf16, bool allow_idx);
int check_layout(const char* fn, const char* name, const gdr_tensor* t, int64_t mult);
int check_index_vec(const char* fn, const char* name, const gdr_tensor* t, int64_t n);
int check_work_dtype(const char* fn, const char* name, const gdr_tensor* t, int32_t work);

// The checks of one call, on its device index vectors (nullptr: absent).
struct IndexCheck {
    const gdr_tensor* offsets = nullptr;
    int64_t total_tokens = 0;
    const gdr_tensor* slots = nullptr;
    int64_t num_slots = 0;
    const gdr_tensor* ring_idx = nullptr;
    int64_t ring_rows = 0, ring_len = 0;
    const gdr_tensor* accepted = nullptr;
};

int run_debug_check(const char* fn, int64_t rows, const IndexCheck& c, void* stream);

float resolve_scale(float scale, int64_t K);
int hip_status(const char* fn, hipError_t e);
const uint32_t* as_u32(const gdr_tensor* t);

// Defined in gdr_block_api.cpp.
int check_distinct(const char* fn, const char* name, const gdr_tensor* t);
int check_workspace(const char* fn, const gdr_tensor* ws, int64_t need);
int check_grid(const char* fn, int64_t blocks, int64_t threads);
int no_alias(const char* fn, const gdr_tensor* out, const char* name,
             std::initializer_list<const gdr_tensor*> ins);
int done();

}  // namespace gdr
