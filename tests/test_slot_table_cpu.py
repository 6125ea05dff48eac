"""What the library remembers of kernels' occupancy (csrc/slot_table.h), compiled for the host: every entry of many
thousands is found again, and entries that differ in one field are different ones. A table that filled up would have every
later call look its kernel up anew."""
import ctypes as C
import os
import subprocess

import pytest

from tests.conftest import ROOT

SOURCE = """
#include "slot_table.h"
static p24::SlotTable table;
extern "C" int find(const void* kern, size_t smem, int dev, int threads, int ranks) {
  return table.find(p24::SlotKey{kern, smem, dev, threads, ranks});
}
extern "C" void put(const void* kern, size_t smem, int dev, int threads, int ranks, int slots) {
  table.put(p24::SlotKey{kern, smem, dev, threads, ranks}, slots);
}
"""


@pytest.fixture(scope="module")
def table(tmp_path_factory):
    d = tmp_path_factory.mktemp("slots")
    src, lib = os.path.join(d, "slots.cpp"), os.path.join(d, "slots.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    csrc = os.path.join(ROOT, "semi_structured_sparse_prune24_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{csrc}", src, "-o", lib], check=True)
    so = C.CDLL(lib)
    so.find.argtypes = [C.c_void_p, C.c_size_t, C.c_int, C.c_int, C.c_int]
    so.put.argtypes = so.find.argtypes + [C.c_int]
    return so


def test_every_entry_is_kept(table):
    keys = [(0x1000 + 16 * (i % 40), 1024 * (i // 40), i % 3, 32 + 32 * (i % 32), 1 << i % 4) for i in range(20000)]
    assert len(set(keys)) == len(keys)
    assert all(table.find(*k) == 0 for k in keys)
    for n, k in enumerate(keys):
        table.put(*k, 1 + n)
    assert all(table.find(*k) == 1 + n for n, k in enumerate(keys))


def test_every_field_counts(table):
    key = (0x9000, 4096, 0, 256, 1)
    table.put(*key, 608)
    assert table.find(*key) == 608
    for at, v in enumerate((0x9010, 4112, 1, 288, 2)):
        assert table.find(*(v if i == at else x for i, x in enumerate(key))) == 0


def test_the_library_uses_it():
    api = open(os.path.join(ROOT, "semi_structured_sparse_prune24_gb300", "csrc", "p24_api.cu")).read()
    body = api[api.index("cudaError_t row_kernel_slots("):]
    assert "SlotTable" in body[:body.index("\n}\n")]
