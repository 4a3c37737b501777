"""The rule for a compaction's cluster sizes, compiled for the host: what a context cannot
hold is never asked for, and where it holds all sizes the rule's own choice stands."""
import ctypes as C
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_59_gb300", "csrc")


@pytest.fixture(scope="module")
def ctas(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("clusters")
    src, lib = at / "rule.cpp", at / "rule.so"
    src.write_text('#include "compact_clusters.h"\nextern "C" int ctas(long long u, int s, long long k, long long n, int t, int l) '
                   "{ return pa_compact_ctas(u, s, k, n, t, l); }\n")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    f = C.CDLL(str(lib)).ctas
    f.argtypes = [C.c_longlong, C.c_int, C.c_longlong, C.c_longlong, C.c_int, C.c_int]
    return f


def test_no_cluster_is_larger_than_the_context_holds(ctas):
    rng = random.Random(1)
    for _ in range(20000):
        units, sms, tokens = rng.choice([2, 4, 16, 32, 100, 5000]), rng.choice([1, 8, 20, 76, 152]), rng.choice([128, 256, 512])
        seqs = rng.randint(1, units)
        kept = int(2 ** rng.uniform(0, 22))
        whole = ctas(units, sms, kept, seqs, tokens, 16)
        for largest in (1, 2, 5, 8, 11, 16):
            got = ctas(units, sms, kept, seqs, tokens, largest)
            assert 1 <= got <= largest
            assert got == whole if whole <= largest else got == largest


def test_sizes_of_one_document_and_of_batches(ctas):
    assert ctas(16, 152, 78643, 1, 128, 16) == 12      # 8 KV heads, K and V, on 152 SMs
    assert ctas(16, 152, 78643, 1, 128, 8) == 8
    assert ctas(8, 152, 50000, 4, 128, 16) == 16
    assert ctas(512, 152, 60000, 32, 128, 16) == 1     # enough units for every SM
    assert ctas(16, 152, 100, 1, 128, 16) == 1         # one step's tokens
