"""Launches of the attention calls at the largest sizes that they accept, on a machine without
a GPU (see attn_launch_probe.cpp): none that HIP refuses, and together all of the work."""
import os
import subprocess

import pytest

import rht_bit_block_amd as U

HERE = os.path.dirname(os.path.abspath(__file__))
pytestmark = pytest.mark.skipif(not os.path.exists(U.LIB_PATH), reason="library not built")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("probe") / "attn_launch_probe")
    subprocess.run(["g++", "-O1", "-rdynamic", os.path.join(HERE, "attn_launch_probe.cpp"), "-o", exe, "-ldl"], check=True)

    def call(fn, *args):
        """(status, [(kernel, grid x y z, block x)])"""
        r = subprocess.run([exe, U.LIB_PATH, fn, *(str(int(a)) for a in args)], capture_output=True, text=True, check=True)
        lines = [x.split() for x in r.stdout.splitlines()]
        assert not [x for x in lines if x[0] == "refused"], [x for x in lines if x[0] == "refused"][:2]
        return int(lines[-1][1]), [(x[1], [int(v) for v in x[2:5]], int(x[5])) for x in lines if x[0] == "launch"]

    return call


# T, B, heads, key heads, D
SIZES = [(1, 1, 1, 1, 128), (1 << 30, 1, 1, 1, 8), (1 << 30, 1 << 20, 2, 2, 64), (1 << 24, 1 << 20, 1024, 1, 128), (1 << 22, 3, 1024, 1024, 64),
         (100, 1 << 20, 1024, 8, 96)]


@pytest.mark.parametrize("T,B,heads,kv,D", SIZES)
def test_attention(probe, T, B, heads, kv, D):
    tiles = T // 128 + B   # as many tiles as B sequences of T rows can have
    st, got = probe("attn_fwd", T, B, heads, kv, D, 16)
    assert st == U.UFP4_OK and all("k_attn_fwd" in x[0] for x in got)
    assert sum(x[1][0] for x in got) == tiles * heads
    st, got = probe("attn_bwd", T, B, heads, kv, D, 16)
    assert st == U.UFP4_OK
    assert sum(x[1][0] for x in got if "k_attn_dq" in x[0]) == tiles * heads
    assert sum(x[1][0] for x in got if "k_attn_dkv" in x[0]) == tiles * kv
    names = ["dq" if "k_attn_dq" in x[0] else "dkv" for x in got]
    assert names == sorted(names, reverse=True)   # dq leaves what dkv reads


@pytest.mark.parametrize("T,B,heads,kv,D", [(1, 1, 1, 1, 128), (1 << 30, 1 << 20, 1, 1, 16), (1 << 28, 7, 8, 8, 128), (1 << 20, 1 << 20, 1024, 1024, 64)])
def test_cache(probe, T, B, heads, kv, D):
    for fn, kernel in (("kv_write", "k_kv_write"), ("kv_read", "k_kv_read")):
        st, got = probe(fn, T, B, heads, kv, D, 16)
        assert st == U.UFP4_OK and got and all(kernel in x[0] for x in got)
        assert sum(x[1][0] * x[2] for x in got) >= T * (D // 16)
        assert all(x[1][1] <= 2 * kv for x in got)
    st, got = probe("kv_attn", T, B, heads, kv, D, 64)
    assert st == U.UFP4_OK and ["k_kv_attn" in x[0] for x in got] == [True, False] and "k_kv_join" in got[1][0]
