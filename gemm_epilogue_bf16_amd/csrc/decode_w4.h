// Launch interface of the 4-bit-weight decode kernel (decode_w4.hip).  Internal
// to the library, like kernels.h; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fmlp {

// One decode layer (M <= 16 tokens) with 4-bit weights [N, K] and bf16 scales
// (and zero points) [N, K / G]: W[n, k] = s (q - z), z = 8 where z0 is null;
// G = 32, 64 or 128 and K % G == 0.  With q1 set it is the gate+up layer
// y = act(x W0^T) * (x W1^T) (z0 and z1 both null or both set), else
// y = act(x W0^T + bias).  One launch,
// up to three where the activations are large.
struct W4Layer {
  const uint16_t* x;     // [M, K] bf16
  const uint8_t* q0;     // [N, K / 2], code 2j in the low half of byte j
  const uint16_t* s0;    // [N, K / G] bf16
  const uint16_t* z0;    // [N, K / G] bf16 or nullptr
  const uint8_t* q1;     // gate+up: the up weights, or nullptr
  const uint16_t* s1;
  const uint16_t* z1;
  const uint16_t* bias;  // [N] or nullptr (ungated only)
  uint16_t* y;           // [M, N] bf16
  int64_t K, N;
  int G;
  int act;               // Act; for a gated layer, the gate's activation
  uint8_t* scratch;      // decode_w4_scratch_bytes of device memory, or nullptr where that is 0
  uint8_t* records;      // (set by the launcher)
};

// Scratch of a call: activations in operand form where a block does not make
// them itself, and the k slices' sums where they do not all fit in LDS.
size_t decode_w4_scratch_bytes(int64_t M, int64_t K, int64_t N, int G, bool dual);
// cus: the device's compute units (the persistent grid's size).
hipError_t launch_decode_w4(const W4Layer& L, int M, int cus, hipStream_t s);

}  // namespace fmlp
