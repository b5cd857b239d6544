// Host helpers of the C ABI's implementation files (defined in api.hip): the calling thread's error
// text, the device check, the launch log and the layout rules that several entry points share.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "tbg.h"

namespace tbg {

// Records the detail tbg_last_error() returns on this thread and passes the status through.
tbg_status fail(tbg_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// A usable device: the current HIP device must be gfx950.  Checked once per device id, which
// also records the device's compute-unit count (returned through num_cus when given).
tbg_status check_device(int* num_cus = nullptr);

// TBG_LOG set to anything but "" or "0": every GEMM and convolution call reports the kernel
// configuration it launches on stderr (read once per process).
void log_choice(const char* fmt, ...) __attribute__((format(printf, 1, 2)));

// Whether the epilogue may store whole 16-byte pieces of C's rows (8-byte pieces in the scaled
// 16-bit path): gfx9's multi-dword memory instructions need only dword-aligned addresses, so C's
// base and its row pitch in bytes must be multiples of 4 (every fp32 C at a 4-byte aligned base;
// a 16-bit C when ldc is even).  Otherwise the epilogue stores element by element.
int rows_dword_aligned(const void* C, int64_t ldc, int elsize);

// Where a call's repacked operands go in the caller's workspace.  A workspace of at least twice
// the need (each half 256-byte aligned) is used by halves, alternately from call to call (one
// counter for the process): a repack that overwrites the copy which the previous product has
// just read runs much slower on MI355X (the 3001×2049×777 operands: ≈8.5 µs, against ≈4.7 µs
// into the other half; kernel trace), and consecutive products usually share one workspace.
// The half only moves where the repack lands, never what the product computes.
uint8_t* repack_area(void* workspace, size_t workspace_bytes, size_t need);

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

}  // namespace tbg
