"""What the library launches, recorded on the host: every shape that a call accepts has to reach a
kernel instance that is made for it.

A small library that stands in for the runtime's launch is loaded before libwq in a process of its
own; nothing runs on a GPU, and no pointer is followed."""

import json
import os
import re
import subprocess
import sys

import pytest

import weight_only_quantized_gemm_amd as wq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RECORDER = r"""
#include <cstddef>
#include <cstdio>
#include <map>
#include <string>
struct dim3 { unsigned x, y, z; };
static std::map<const void*, std::string> names;
static std::string launches;
static dim3 grid_, block_;
static size_t shared_;
static void* stream_;
extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* handle; return &handle; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(...) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*,
                           void*, void*, int*) { names[host] = name; }
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, void* stream) {
  grid_ = grid, block_ = block, shared_ = shared, stream_ = stream;
  return 0;
}
int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, void** stream) {
  *grid = grid_, *block = block_, *shared = shared_, *stream = stream_;
  return 0;
}
int hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t, void*) {
  char sizes[64];
  std::snprintf(sizes, sizeof sizes, " %u %u %u\n", grid.x, grid.y, block.x);
  launches += names[f] + sizes;
  return 0;
}
int hipGetLastError() { return 0; }
const char* take_launches() {
  static std::string out;
  out = launches;
  launches.clear();
  return out.c_str();
}
}
"""

# One line of JSON for each line of it on stdin: a call's status and its launches.
WALK = r"""
import ctypes, json, sys
fake = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)
fake.take_launches.restype = ctypes.c_char_p
sys.path.insert(0, sys.argv[2])
import weight_only_quantized_gemm_amd as wq
P, L = 1 << 20, wq.lib()
for line in sys.stdin:
    c = json.loads(line)
    d, group, hkv, hq, flags = c["d"], c["group"], c["hkv"], c["hq"], c["flags"]
    groups = d // group
    cache = wq.wq_kv_cache(k=P, v=2 * P, page_stride=16 * hkv * d, slot_stride=hkv * d, head_stride=d,
                           num_pages=9, page_size=16, kv_heads=hkv, head_dim=d)
    pairs = wq.wq_kv_pairs(k=3 * P, v=4 * P, page_stride=16 * hkv * groups,
                           slot_stride=hkv * groups, head_stride=groups, group_size=group)
    need = ctypes.c_size_t(0)
    assert L.wq_paged_attention4_workspace_bytes(c["batch"], hq, hkv, d, group, c["max_len"], 0,
                                                 ctypes.byref(need)) == 0, c
    a = wq.versioned(wq.wq_attn4_args, cache=cache, pairs=pairs, q=5 * P, out=6 * P, block_table=7 * P,
                     lens=8 * P, workspace=9 * P, workspace_bytes=need.value, batch=c["batch"],
                     q_heads=hq, max_len=c["max_len"], table_stride=c["max_len"] // 16 + 1,
                     ldq=hq * d, ldo=hq * d, scale=0.1, flags=flags)
    status = L.wq_paged_attention4(ctypes.byref(a))
    print(json.dumps([status, need.value, fake.take_launches().decode().splitlines()]))
"""


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    at = tmp_path_factory.mktemp("launches")
    (at / "recorder.cc").write_text(RECORDER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", str(at / "recorder.cc"), "-o",
                    str(at / "recorder.so")], check=True)
    return str(at / "recorder.so")


def walk(recorder, cases):
    done = subprocess.run([sys.executable, "-c", WALK, recorder, ROOT], capture_output=True, text=True,
                          input="\n".join(map(json.dumps, cases)), timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
    return list(zip(cases, map(json.loads, done.stdout.splitlines()), strict=True))


def test_every_accepted_shape_of_the_4_bit_attention_has_its_kernel(recorder):
    """Every head size with every group of it, query heads to a KV head from one to more than an
    instance takes, odd and even numbers of KV heads, sequences whole and cut."""
    cases = [dict(d=d, group=group, hkv=hkv, hq=hkv * per, batch=batch, max_len=max_len, flags=flags)
             for d in range(16, 257, 8) for group in {d, 32, 64, 128} if d % group == 0
             for hkv in (1, 2, 3, 8) for per in (1, 2, 3, 4, 5, 8, 16, 17)
             for batch, max_len in ((1, 100), (3, 5000)) for flags in (0, wq.WQ_FLAG_BF16)]
    seen = set()
    for c, (status, need, launches) in walk(recorder, cases):
        assert status == 0 and len(launches) == (2 if need else 1), (c, launches)
        at = re.search(r"attn4_kernelILb(\d)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb(\d)E", launches[0])
        assert at, (c, launches)
        bf16, w, groups, sets, kv_heads, full = (int(x) for x in at.groups())
        d, per = c["d"], c["hq"] // c["hkv"]
        assert bf16 == (c["flags"] != 0) and groups == d // c["group"], (c, launches)
        assert full == (d == 32 * w) and 32 * w == min(x for x in (64, 96, 128, 192, 256) if x >= d)
        padded = min(x for x in (1, 2, 4, 8) if x >= groups)
        heads = 16 * sets // padded  # query heads of a work-group
        assert kv_heads == 1 or (sets == 1 and 2 * per <= heads), (c, launches)
        units = -(-c["hkv"] // kv_heads) * -(-kv_heads * per // heads)
        grid, _, threads = (int(x) for x in launches[0].split()[1:])
        assert grid % units == 0 and threads == 256, (c, launches)
        assert need or grid in (c["batch"] * units, -(-c["batch"] // 8) * 8 * units), (c, launches)
        if need:
            shift = heads.bit_length() - 1
            assert f"attn_join_kernelILb{bf16}ELi{shift}E" in launches[1], (c, launches)
            assert launches[1].split()[1:3] == [str(c["hq"]), str(c["batch"])]
        seen.add(at.group(0))
    assert len(seen) > 80  # most instances that there are
