"""The C entry points of the rotation and the 8-bit cache over stand-ins for the device and
the launches: plans, workspace sizes and what happens where the host fails."""
from __future__ import annotations

import os
import subprocess

import pytest

from token_decode_attention_gb300 import build

STANDINS = r"""
#include "dattn.h"
#include "dattn_internal.h"
#include <cstdio>
#include <cstdlib>
#include <new>
#include <string>
#include <vector>

static std::string g_message;
static int g_launches = 0, g_occupancy = 0;
static bool g_no_memory = false, g_no_message = false;

namespace dattn {
int set_last_error(int status, const char *m) {
    if (g_no_message) throw std::bad_alloc();
    g_message = m;
    return status;
}
int device_facts(DeviceFacts *out) {
    if (g_no_memory) throw std::bad_alloc();
    static unsigned word;
    *out = DeviceFacts{152, 232448, &word};
    return DATTN_OK;
}
cudaError_t decode_q8_configure(int) { return cudaSuccess; }
cudaError_t decode_q8_max_clusters(int, int, bool, int, int cluster, int *n) {
    ++g_occupancy;
    *n = 304 / cluster;
    return cudaSuccess;
}
cudaError_t launch_decode_q8(const Q8DecodeArgs &, int, int, int, int, cudaStream_t) { ++g_launches; return cudaSuccess; }
cudaError_t launch_combine(const CombineArgs &, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_rope(const RopeArgs &, int, int, cudaStream_t) { ++g_launches; return cudaSuccess; }
cudaError_t launch_append_q8(const Q8AppendArgs &, int, int, cudaStream_t) { ++g_launches; return cudaSuccess; }
}
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char *cudaGetErrorName(cudaError_t) { return ""; }
const char *cudaGetErrorString(cudaError_t) { return ""; }
}
// allocations that are alive
static long long g_alive = 0;
void *operator new(size_t n) {
    void *p = std::malloc(n);
    if (!p) throw std::bad_alloc();
    ++g_alive;
    return p;
}
void operator delete(void *p) noexcept { if (p) --g_alive, std::free(p); }
void operator delete(void *p, size_t) noexcept { operator delete(p); }
static char *const A = reinterpret_cast<char *>(0x10000);
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s (%s)\n", __LINE__, #x, g_message.c_str()); return 1; } } while (0)
"""


@pytest.fixture
def run(tmp_path):
    def go(body: str) -> None:
        src, exe = tmp_path / "t.cpp", tmp_path / "t"
        src.write_text(STANDINS + "int main() {\n" + body + "\nreturn 0;\n}\n")
        cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
        subprocess.run(["g++", "-O1", "-std=c++17", f"-I{build.CSRC}", f"-I{build.INCLUDE}", f"-I{cuda}",
                        str(src), os.path.join(build.CSRC, "q8_api.cpp"), "-o", str(exe)], check=True)
        r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout + r.stderr
    return go


def test_queries_take_a_wide_table_over_a_small_pool(run):
    # 2048 sequences of up to 2^20 positions in a pool of 8 pages: the capacities add up to 2^31
    run("""
    size_t bytes = 0;
    dattn_plan plan;
    CHECK(dattn_decode_q8_workspace_bytes(2048, 2, 1, 16, 1 << 20, 0, &bytes) == DATTN_OK);
    CHECK(dattn_decode_q8_plan(2048, 2, 1, 16, 1 << 20, 0, &plan) == DATTN_OK);
    CHECK(plan.workspace_bytes == bytes);
    CHECK(dattn_decode_paged_q8(A, A, A, (float *)A, (float *)A, A, DATTN_KV_E4M3, 16, 2048, 2, 1, 16, 256, 4096, 8,
                                (int32_t *)A, (uint32_t *)A, A, bytes, 0, nullptr) == DATTN_OK);
    CHECK(bytes == 0 || dattn_decode_paged_q8(A, A, A, (float *)A, (float *)A, A, DATTN_KV_E4M3, 16, 2048, 2, 1, 16, 256,
                                              4096, 8, (int32_t *)A, (uint32_t *)A, A, bytes - 1, 0, nullptr) ==
                              DATTN_ERR_WORKSPACE);
    // the calls themselves count the rows that there are
    CHECK(dattn_decode_q8(A, A, A, (float *)A, (float *)A, A, DATTN_KV_E4M3, 16, 2048, 2, 1, 16, 1 << 20, (uint32_t *)A, A,
                          size_t(1) << 40, 0, nullptr) == DATTN_ERR_UNSUPPORTED);
    CHECK(dattn_decode_paged_q8(A, A, A, (float *)A, (float *)A, A, DATTN_KV_E4M3, 16, 1, 2, 1, 16, 256, 4096, 1LL << 24,
                                (int32_t *)A, (uint32_t *)A, A, size_t(1) << 40, 0, nullptr) == DATTN_ERR_UNSUPPORTED);
    CHECK(g_launches == 1);
    // what no call takes is refused by the queries too
    CHECK(dattn_decode_q8_workspace_bytes(2048, 2, 1, 16, 0, 0, &bytes) == DATTN_ERR_INVALID_ARG);
    CHECK(dattn_decode_q8_workspace_bytes(1, 1 << 30, 1 << 30, 16, 64, 0, &bytes) == DATTN_ERR_UNSUPPORTED);
""")


def test_a_failure_of_the_host_has_its_own_message(run):
    run("""
    dattn_rope_params r{64, 0, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, 1.0};
    g_message = "of an earlier call";
    g_no_memory = true;
    CHECK(dattn_rope(A, A, DATTN_F16, 4, 2, 64, 128, 128, (uint32_t *)A, &r, 0, nullptr) == DATTN_ERR_CUDA);
    CHECK(g_message.find("earlier") == std::string::npos && !g_message.empty());
    g_message = "of an earlier call";
    size_t bytes = 0;
    CHECK(dattn_decode_q8_workspace_bytes(1, 2, 1, 16, 64, 0, &bytes) == DATTN_ERR_CUDA);
    CHECK(g_message.find("earlier") == std::string::npos && !g_message.empty());
    CHECK(g_launches == 0);
    // nor does a failure to keep the message leave the entry
    g_no_message = true;
    CHECK(dattn_decode_q8_workspace_bytes(1, 2, 1, 16, 64, 0, &bytes) == DATTN_ERR_CUDA);
""")


def test_plans_are_kept_for_a_bounded_number_of_shapes(run):
    # a process that sees a new capacity at every step keeps no more than some of them
    run("""
    dattn_plan first, again;
    CHECK(dattn_decode_q8_plan(1, 8, 8, 64, 500, 0, &first) == DATTN_OK);
    const long long before = g_alive;
    for (int s = 1; s <= 20000; ++s) {
        dattn_plan p;
        CHECK(dattn_decode_q8_plan(2, 8, 2, 128, s, 0, &p) == DATTN_OK);
    }
    CHECK(g_alive - before < 2000);
    const int asked = g_occupancy;
    CHECK(dattn_decode_q8_plan(2, 8, 2, 128, 20000, 0, &again) == DATTN_OK);
    CHECK(g_occupancy == asked);   // the latest is kept
    CHECK(dattn_decode_q8_plan(1, 8, 8, 64, 500, 0, &again) == DATTN_OK);
    CHECK(first.partitions == again.partitions && first.cluster_size == again.cluster_size &&
          first.workspace_bytes == again.workspace_bytes && first.heads_per_cta == again.heads_per_cta);
""")


def test_overlapping_tensors_are_refused_and_neighbours_launched(run):
    # rows of 2 x 64 f16
    run("""
    dattn_rope_params r{8, 0, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, 1.0};
    auto rope = [&](char *x, long long xs, char *out, long long os, long long T) {
        return dattn_rope(x, out, DATTN_F16, T, 2, 64, xs, os, (uint32_t *)A, &r, 0, nullptr);
    };
    CHECK(rope(A, 256, A + 256, 256, 4) == DATTN_OK);
    CHECK(rope(A + 256, 256, A, 256, 4) == DATTN_OK);
    CHECK(rope(A, 136, A, 128, 1) == DATTN_OK);
    CHECK(rope(A, 128, A + 1024, 128, 4) == DATTN_OK);
    CHECK(rope(A, 128, A, 128, 4) == DATTN_OK);
    CHECK(g_launches == 5);
    CHECK(rope(A, 128, A + 16, 128, 4) == DATTN_ERR_INVALID_ARG);
    CHECK(rope(A, 256, A + 240, 256, 4) == DATTN_ERR_INVALID_ARG);
    CHECK(rope(A, 136, A, 128, 4) == DATTN_ERR_INVALID_ARG);
    auto append = [&](char *q, long long qs, char *qo) {
        return dattn_rope_append_q8(q, A, A, qo, A, A, (float *)A, (float *)A, DATTN_KV_E4M3, 16, 4, 4, nullptr, qs, 64, 64,
                                    2, 1, 64, 64, &r, (uint32_t *)A, nullptr);
    };
    CHECK(append(A, 128, A) == DATTN_OK && append(A, 128, A + 1024) == DATTN_OK);
    CHECK(g_launches == 7);
    CHECK(append(A, 128, A + 16) == DATTN_ERR_INVALID_ARG);
    CHECK(append(A, 256, A) == DATTN_ERR_INVALID_ARG && append(A, 256, A + 256) == DATTN_ERR_INVALID_ARG);
    CHECK(g_launches == 7);
""")
