// ops_stub.cpp, with what the last rotation of np_rope_apply turns its pairs by: compiled by tests/test_rope_turns.py.
#include "ops_stub.cpp"

extern "C" {
int stub_turns(uint64_t* out) {
    for (int i = 0; i < g_rope.rope.rot / 2; ++i) out[i] = g_rope.rope.turns[i];
    return g_rope.rope.rot / 2;
}
}
