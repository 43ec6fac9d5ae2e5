// pkv_invoke: a call's arguments from one array of 64-bit words, each
// converted to the parameter it stands for.
#include <cstdint>
#include <cstring>
#include <tuple>
#include <type_traits>
#include <utility>

#include "pkv.h"

namespace {

template <typename T>
bool take(const unsigned char* at, T& v) {
    if constexpr (std::is_pointer_v<T>) {
        uint64_t w;
        std::memcpy(&w, at, 8);
        v = reinterpret_cast<T>(static_cast<uintptr_t>(w));
    } else if constexpr (std::is_floating_point_v<T>) {
        double w;
        std::memcpy(&w, at, 8);
        v = static_cast<T>(w);
    } else if constexpr (std::is_integral_v<T> && sizeof(T) == 8) {
        std::memcpy(&v, at, 8);
    } else {                                  // int and enumerations
        int64_t w;
        std::memcpy(&w, at, 8);
        if (w < INT32_MIN || w > INT32_MAX) return false;
        v = static_cast<T>(w);
    }
    return true;
}

template <typename... A, size_t... I>
pkv_status spread(pkv_status (*call)(A...), const unsigned char* words, std::index_sequence<I...>) {
    std::tuple<A...> args;
    if (!(take(words + 8 * I, std::get<I>(args)) && ...)) return PKV_ERR_INVALID_ARG;
    return call(std::get<I>(args)...);
}

template <typename... A>
pkv_status run(pkv_status (*call)(A...), const void* words) {
    return spread(call, static_cast<const unsigned char*>(words), std::index_sequence_for<A...>{});
}

}  // namespace

extern "C" pkv_status pkv_invoke(int call, const void* words) {
    if (words == nullptr) return PKV_ERR_INVALID_ARG;
    switch (call) {
        case PKV_CALL_DECODE_WINDOW: return run(pkv_paged_attention_decode_window, words);
        case PKV_CALL_PREFILL_WINDOW: return run(pkv_paged_attention_prefill_window, words);
        case PKV_CALL_KV4_WRITE: return run(pkv_paged_kv4_write, words);
        case PKV_CALL_KV4_READ: return run(pkv_paged_kv4_read, words);
        case PKV_CALL_DECODE_KV4: return run(pkv_paged_attention_decode_kv4, words);
        case PKV_CALL_DECODE_SCORED: return run(pkv_token_attention_decode_scored, words);
        case PKV_CALL_EVICT: return run(pkv_evict_tokens, words);
        case PKV_CALL_ROTARY_WRITE: return run(pkv_rotary_kv_write, words);
        case PKV_CALL_PROMPT: return run(pkv_prompt_attention, words);
        case PKV_CALL_DECODE_SHARED: return run(pkv_paged_attention_decode_shared, words);
    }
    return PKV_ERR_INVALID_ARG;
}
