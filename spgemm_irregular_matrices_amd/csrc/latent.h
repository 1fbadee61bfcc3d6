// Launchers and shared types of latent attention (include/spgemm_cache.h).
#pragma once

#include "../../include/spgemm_cache.h"
#include "attention_paged.h"

namespace sg {

// Absorbed: k, k_page, k_slot, k_shift place a token's latent row, whose first
// s.dim values are its value. Expanded: a head's keys and values lie in the
// workspace, one row per place of the table (or per sequence and place), and
// the latent row gives the keys' last values.
struct LatentArgs : PagedArgs {
    int key_dim = 0;      // values of a query
    int made_dim = 0;     // expanded: those that the weights make
    int rope_at = 0;      // expanded: bytes from a latent row's start to its last values
    char* made_k = nullptr;  // [head][row][2][made_dim]: rounded values, and what that leaves
    char* made_v = nullptr;  // [head][row][2][s.dim]
    int64_t made_rows = 0;
    int64_t made_step = 0;   // rows per sequence; 0: a row per place of the table
};
constexpr int kAbsorbedEvenSeqs = 1024;  // sequences that are cut evenly
constexpr int kAbsorbedKeys = 64;  // keys per tile of the absorbed form
int latent_tile_rows(const LatentArgs& a, bool absorbed);
void latent_attention(const LatentArgs& a, bool absorbed, hipStream_t st);

struct ExpandArgs {
    LatentArgs a;
    AttnRows wk, wv;     // row: head, head: the key's or value's index; bytes
    int latent_dim = 0;
};
void latent_expand(const ExpandArgs& e, hipStream_t st);

}  // namespace sg
