// Sizes that the projection's kernels and plans share.
#pragma once

namespace tts {
namespace {

constexpr int kM = 128;               // rows of a product's first operand a tile
constexpr int kRowBytes = 128;        // bytes of K a swizzled row holds

}  // namespace
}  // namespace tts
