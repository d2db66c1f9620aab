// prompt.cuh -- attention over whole prompts: what the plan (prompt.cu) and the kernels
// (prompt_attn.cuh) share.
//
// The work is a list of items, a piece of one prompt's tokens and a key head each.  The rows
// of an item are (token, query head of the group) pairs, row = token * G + head, so that
// the keys and values of a tile are read once for all heads of their group.
#pragma once

#include <cuda.h>

#include "tensor.cuh"

namespace sv {

constexpr int PROMPT_KEYS = 128;  // keys of a tile
constexpr int PROMPT_ROWS = 128;  // rows of a row tile; an item has two

// tokens of a row tile
__host__ __device__ inline int prompt_tokens(int G) { return PROMPT_ROWS / G; }

// One piece of a prompt: up to 2 * prompt_tokens(G) tokens.
struct __align__(16) PromptItem {
    int q0;     // its first token, packed
    int n;      // its tokens
    int k0;     // the prompt's first key, packed
    int last;   // the last key that token q0 sees, in the prompt; token q0 + i sees i more (negative: none)
    int m;      // the prompt's keys
    int pad[3];
};

// The plan: a header of 16 words, then the items, the longest first, then prefix sums of
// the prompts' pieces (spec_prompt_plan's own).
struct PromptHead {
    int items, T, M, tokens;  // pieces, packed queries and keys, tokens of a row tile
    int pad[12];
};
inline long long prompt_max_items(int B, long long T, int G) {
    const long long each = 2 * prompt_tokens(G);
    return T / each + (T < B ? T : B);  // every prompt that has tokens adds one piece at most
}

struct PromptArgs {
    const PromptHead* plan;
    void* out;
    float* lse;
    const void* v;
    long long v_token, v_head;
    int T, M, Hq, Hkv, G, D, tokens;
    int window;  // keys that a query sees at most (0: all)
    float c;     // scale * log2(e)
    int32_t* status;
};

struct PromptLaunch {
    CUtensorMap mq, mk, mv, mo;
    PromptArgs A;
    long long items;  // of all heads, at most
    int sms;
    cudaStream_t st;
};
cudaError_t launch_prompt_bf16(const PromptLaunch& L);
cudaError_t launch_prompt_f16(const PromptLaunch& L);

}  // namespace sv
