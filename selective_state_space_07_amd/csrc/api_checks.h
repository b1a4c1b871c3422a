// What the C-ABI entry points of libmamba_scan share (defined in
// mamba_scan_api.cpp): the thread's error detail, pointer and extent checks,
// the aliasing rules, the device check and the call counter. Host code only;
// nothing here makes a HIP call except check_device.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>
#include <string>

namespace mscan {
namespace api {

// Record `fmt` as the thread's last error and return `status`.
int fail(int status, const char* fmt, ...);
// Clear the thread's last error and return MAMBA_OK.
int ok();
// The thread's last error, for size queries that leave it as it was.
std::string& last_error();
// Count one successful launch.
void count_call();

size_t io_size(int32_t io_dtype);

struct Range {
  const char* name;
  uintptr_t lo, hi;  // [lo, hi)
};
Range range(const char* name, const void* p, size_t bytes);
bool overlaps(const Range& a, const Range& b);
bool aligned(const void* p, size_t a);

// Whether the product of non-negative 32-bit extents stays below 2^31,
// evaluated without overflow (each partial product is checked before the
// next factor, so it never exceeds 2^62).
bool below_2_31(std::initializer_list<int64_t> factors);

// Outputs may not overlap inputs, except that a state output may coincide
// exactly with its own state input. Outputs may not overlap one another.
int check_alias(const Range* ins, int n_in, const Range* outs, int n_out, const Range* pair_in,
                const Range* pair_out, int n_pairs);

// The current device is a gfx950.
int check_device();

}  // namespace api
}  // namespace mscan
