// The 4-bit cache format: where a block's codes, scales and zeros lie.
//
// A block of bs tokens holds, for each K/V head on its own, bs * (d/2 + d/8)
// consecutive bytes: bs * d 4-bit codes, then bs * d/32 scales and as many
// zeros in fp16.  A group is 32 consecutive values of a row; G = d / 32.
// value = (zero + scale * code) * tensor scale.  The bytes of one head of one
// block are one bulk copy, and the codes lie in the order the decode's
// matrix instructions take them, so a lane reads its operands with one
// 16-byte load (8-byte for d = 64) free of bank conflicts, and unpacks them
// with one AND per two values, no shuffle.  (Element e of token t; 32-bit
// words of 8 codes, code j in bits 4j.)
//
//   K: word ((t * 4 + e % 32 / 8) * G + e / 32), code e % 8.
//      A lane of the logits product holds, for its token, the four-lane
//      group's quarter of every group: one word per group.
//   V: word ((t / 8 * 8 + e % 32 / 4) * 4 + t / 2 % 4) * G + e / 32,
//      code 4 * (t % 2) + e % 4.  Two tokens share a word, since the product
//      over tokens takes two of them side by side in a register.
//   scales, zeros of K: [token][group]; of V: [token / 2][group][token % 2].
#pragma once

#include "pkv_common.cuh"

namespace pkv {

constexpr int kKv4Group = 32;
constexpr float kKv4Max = 65504.f;       // largest magnitude of a scaled value: fp16's

__host__ __device__ constexpr int kv4_head_bytes(int bs, int d) { return bs * (d / 2 + d / 8); }

template <int D>
struct Kv4 {
    static constexpr int G = D / kKv4Group;
    static __device__ __forceinline__ int codes(int bs) { return bs * (D / 2); }
    static __device__ __forceinline__ int k_word(int t, int e) { return (t * 4 + e % 32 / 8) * G + e / 32; }
    static __device__ __forceinline__ int v_word(int t, int e) {
        return ((t / 8 * 8 + e % 32 / 4) * 4 + t / 2 % 4) * G + e / 32;
    }
    // index among the block's scales (or zeros)
    static __device__ __forceinline__ int k_par(int t, int g) { return t * G + g; }
    static __device__ __forceinline__ int v_par(int t, int g) { return (t / 2 * G + g) * 2 + t % 2; }
};

}  // namespace pkv
