"""CPU tests of csrc/gdnt_chain.hpp, how a state travels between tiles: the
header is compiled by g++ as a wave of one lane, the device builtins it uses
replaced by plain C++, and run on chains of words laid out by hand."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHAIN = os.path.join(ROOT, "linear_attention_ssm_gdn_amd", "csrc", "gdnt_chain.hpp")

DEVICE = r"""
#pragma once
#include <cmath>
#include <math.h>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <limits>
#define __device__
#define __forceinline__ inline
#define __all(x) (x)
#define __HIP_MEMORY_SCOPE_AGENT 0
#define __hip_atomic_load(p, order, scope) (*(p))
#define __hip_atomic_store(p, v, order, scope) (*(p) = (v))
#define __builtin_amdgcn_s_sleep(n) ((void)0)
#define GDNT_DEVERR_TIMEOUT 32u
struct Idx { int x; };
static Idx threadIdx{0};
inline float __uint_as_float(uint32_t v) { float f; memcpy(&f, &v, 4); return f; }
inline uint32_t __float_as_uint(float f) { uint32_t v; memcpy(&v, &f, 4); return v; }
namespace gdnt {
constexpr float kTiny = 1.17549435e-38f;
inline void raise(int32_t* err, uint32_t bit) { if (err) *err |= (int32_t)bit; }
}
"""

MAIN = r"""
#include "gdnt_chain.hpp"
#include <cstdio>
#include <cstdlib>
using namespace gdnt;
#define CHECK(c) do { if (!(c)) { printf("line %d: %s\n", __LINE__, #c); exit(1); } } while (0)
constexpr int kTiles = 8;
static uint64_t words[2 * kTiles];
static const Chain chain{words, kTiles};
static const float nan_ = std::numeric_limits<float>::quiet_NaN();

// tiles 0 .. n-1 publish a run each, the first its known end
static void fill(int n) {
    memset(words, 0, sizeof(words));
    for (int t = 0; t < n; ++t) {
        const float a[1] = {t == 0 ? -0.5f : 0.5f}, u[1] = {1.0f + t};
        tell_run<1>(chain, t, t > 0, true, a, u);
    }
}

int main(int argc, char** argv) {
    const char* what = argv[1];
    int32_t err = 0;
    float h[1];
    if (!strcmp(what, "values")) {
        // the state through the runs, at whichever tile it is found: ends 1, 2.5, 4.25, 6.125
        fill(4);
        look_back<1>(chain, 4, -1, 4, h, &err);
        CHECK(h[0] == 6.125f && err == 0);
        chain_store(words + 2, 1u, 4.25f);
        look_back<1>(chain, 4, -1, 4, h, &err);
        CHECK(h[0] == 6.125f && err == 0);
        // a tile with a first row forgets what came before; one that continues hands its end on
        const float begins[1] = {-0.25f}, goes_on[1] = {0.5f}, u[1] = {7.0f};
        hand_on<1>(chain, 4, -1, 4, true, true, goes_on, u, h, &err);
        CHECK(h[0] == 6.125f && words[4] == ((uint64_t)1 << 32 | __float_as_uint(10.0625f)));
        words[4] = 0;
        tell_run<1>(chain, 4, true, true, begins, u);
        hand_on<1>(chain, 4, -1, 4, true, true, begins, u, h, &err);
        CHECK(h[0] == 6.125f && words[4] == ((uint64_t)1 << 32 | __float_as_uint(7.0f)) && err == 0);
        // nothing continues: zero, and nothing is waited for
        hand_on<1>(chain, 6, -1, 6, false, true, goes_on, u, h, &err);
        CHECK(h[0] == 0.0f && err == 0);
    } else if (!strcmp(what, "marks")) {
        // a NaN's sign is not a mark, whichever it is; a mark stays through a join with a NaN run
        for (float v : {nan_, -nan_, 0.0f, 0.5f}) {
            CHECK(marked(v, true) < 0.0f && marked(v, false) > 0.0f);
            CHECK(end_known<1>({marked(v, true)}, true) && !end_known<1>({marked(v, false)}, true));
            float qa = marked(v, false), qu = 1.0f;
            join(marked(0.5f, true), 2.0f, qa, qu);
            CHECK(qa < 0.0f);
        }
        float two[2] = {marked(nan_, false), marked(0.5f, false)}, both[2] = {marked(-nan_, true), marked(0.5f, true)};
        CHECK(!end_known<2>(two, true) && end_known<2>(both, true));
    } else if (!strcmp(what, "timeout")) {
        // tile 2 never publishes: the wait ends, and what follows is no number, here and in the tile after
        fill(2);
        look_back<1>(chain, 3, -1, 3, h, &err);
        CHECK(std::isnan(h[0]) && err == (int32_t)GDNT_DEVERR_TIMEOUT);
        const float a[1] = {0.5f}, u[1] = {1.0f};
        err = 0;
        hand_on<1>(chain, 3, -1, 3, true, true, a, u, h, &err);
        CHECK(std::isnan(h[0]) && err == (int32_t)GDNT_DEVERR_TIMEOUT);
        CHECK((words[3] >> 32) != 0 && std::isnan(__uint_as_float((uint32_t)words[3])));
        look_back<1>(chain, 4, -1, 1, h, nullptr);
        CHECK(std::isnan(h[0]));
    } else {
        return 2;
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    d = tmp_path_factory.mktemp("chain")
    shutil.copy(CHAIN, d)
    (d / "gdnt_device.hpp").write_text(DEVICE)
    (d / "main.cpp").write_text(MAIN)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-w", str(d / "main.cpp"), "-o", str(d / "main")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(d / "main")


@pytest.mark.parametrize("what", ["values", "marks", "timeout"])
def test_the_chain_between_tiles(exe, what):
    r = subprocess.run([exe, what], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
