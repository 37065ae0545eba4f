"""Launches at the largest sizes that the language-model operators accept, on a
machine without a GPU: a small program stands in for the HIP runtime, records
every launch of a call and refuses what HIP refuses (2^32 threads or more in a
grid's dimension).  Pointers are numbers that nobody follows."""
import os
import subprocess

import pytest

import rht_bit_block_amd as U

HERE = os.path.dirname(os.path.abspath(__file__))
P = 1 << 44          # an address; arrays lie 2^44 apart

pytestmark = pytest.mark.skipif(not os.path.exists(U.LIB_PATH), reason="library not built")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("probe") / "launch_probe")
    subprocess.run(["g++", "-O1", "-rdynamic", os.path.join(HERE, "launch_probe.cpp"), "-o", exe, "-ldl"],
                   check=True)

    def call(fn, *args, words=None):
        """(status, [(kernel, grid x y z, block x y z, words of the first argument)]);
        words: part of the names of the kernels whose argument is asked for"""
        env = dict(os.environ)
        if words:
            env["PROBE_WORDS"] = words
        r = subprocess.run([exe, U.LIB_PATH, fn, *(str(int(a)) for a in args)], capture_output=True,
                           text=True, check=True, env=env)
        lines = [x.split() for x in r.stdout.splitlines()]
        assert not [x for x in lines if x[0] == "refused"], [x for x in lines if x[0] == "refused"][:2]
        got = [(x[1], [int(v) for v in x[2:8]], [int(v) for v in x[8:]]) for x in lines if x[0] == "launch"]
        return int(lines[-1][1]), got

    return call


# Places of GluLaunch's fields among its 8-byte words
GATE, UP, ROW, H, GC, GS, DH, DG, DU, DROW, ROWS = 0, 1, 3, 4, 6, 7, 10, 12, 13, 15, 16


def glu_bwd(probe, rows, cols, dtype, drow, again):
    return probe("ufp4_glu_bwd", P, 2 * P, 3 * P, 4 * P, rows, cols, 0, 5 * P, 6 * P, dtype, cols, 7 * P,
                 8 * P, cols, 9 * P if drow else 0, 10 * P if again else 0, cols, 0, words="k_glu")


@pytest.mark.parametrize("rows,cols", [(1 << 26, 32), ((1 << 28) + 3, 1), (1 << 26, 128), (1 << 27, 129),
                                       ((1 << 30) + 7, 0), (1, 1 << 30), (1 << 20, 4096)])
@pytest.mark.parametrize("dtype", [U.UFP4_BF16, U.UFP4_FP32])
def test_glu_backward_with_the_row_factors_gradient(probe, rows, cols, dtype):
    """A wave per row, whatever the row's width; the slices follow one another."""
    st, got = glu_bwd(probe, rows, cols, dtype, True, cols > 0)
    assert st == U.UFP4_OK and got
    at = 0
    for name, g, w in got:
        assert "k_glu_bwd_row" in name
        n = w[ROWS]
        assert g[0] * g[3] >= 64 * n and g[0] * g[3] - 64 * n < 4 * 64
        assert w[DROW] == 9 * P + 4 * at and w[ROW] == 5 * P + 4 * at
        if cols:
            assert w[GC] == P + cols * at and w[GS] == 2 * P + (cols + 31) // 32 * at
            assert w[DH] == 6 * P + (2, 4)[dtype] * cols * at and w[DG] == 7 * P + 2 * cols * at
            assert w[DU] == 8 * P + 2 * cols * at and w[H] == 10 * P + 2 * cols * at
        at += n
    assert at == rows


@pytest.mark.parametrize("rows,cols", [(1 << 26, 32), ((1 << 28) + 3, 1), (1 << 27, 129), (1, 1 << 30)])
def test_glu_forward_and_backward_without_it(probe, rows, cols):
    fwd = probe("ufp4_glu_fwd", P, 2 * P, 1, rows, cols, cols, 0, 3 * P, 4 * P, cols, 5 * P, 6 * P, 7 * P,
                8 * P, 0, words="k_glu")
    chunks = 4 * ((cols + 31) // 32)
    for st, got in (fwd, glu_bwd(probe, rows, cols, 1, False, False)):
        assert st == U.UFP4_OK
        at = 0
        for name, g, w in got:
            n = w[ROWS]
            assert 0 <= g[0] * g[3] - chunks * n < 256
            assert w[ROW] == (3 if "fwd" in name else 5) * P + 4 * at
            assert w[GATE if "fwd" in name else DH] == (P if "fwd" in name else 6 * P) + 4 * cols * at
            at += n
        assert at == rows


# Places of the product's description among its 8-byte words
B_, M_, N_, LDB = 1, 2, 3, 6
W, HID, TG, WS = P, 2 * P, 3 * P, 4 * P


def xent_fwd(probe, T, V, D, words=None):
    return probe("ufp4_linear_xent_fwd", HID, D, W, D, TG, T, V, D, 5 * P, 6 * P, WS, 1 << 62, 0, words=words)


@pytest.mark.parametrize("T,V,D", [(1 << 20, 1 << 20, 64), (1 << 21, 1 << 18, 64), (1 << 21, 1 << 30, 8),
                                   ((1 << 20) + 33, (1 << 22) + 5, 64), (64, 1 << 30, 64), (1, 1 << 30, 8)])
def test_xent_forward(probe, T, V, D):
    """Every token in one launch of the product, whatever T V."""
    st, got = xent_fwd(probe, T, V, D)
    assert st == U.UFP4_OK
    assert ["k_prod" in n for n, _, _ in got] == [True] * (len(got) - 1) + [False]
    wide, tokens = (256, 256) if T > 64 else (128, 64)
    tiles = sum(g[0] for _, g, _ in got[:-1])
    assert tiles == -(-V // wide) * -(-T // tokens)


def test_xent_forward_slices(probe):
    """Slices of tokens follow one another, all with the tile shape that the
    workspace is laid out for, a last one of 33 tokens too."""
    T, V, D = (1 << 20) + 33, 1 << 20, 64
    st, got = xent_fwd(probe, T, V, D, words="k_prod")
    at = 0
    assert st == U.UFP4_OK and len(got) > 2
    for name, g, w in got[:-1]:
        assert name == got[0][0] and w[M_] == V and w[B_] == HID + 2 * D * at and w[LDB] == D
        at += w[N_]
    assert at == T and got[-2][2][N_] == 33


@pytest.mark.parametrize("T,V,D", [(0, 1 << 30, 64), (0, 1 << 21, 1 << 14), (1 << 21, 300, 1 << 13),
                                   (1 << 21, 300, 1 << 17), (1 << 18, 300, 1 << 20), (1, 70000, 1 << 20),
                                   (1 << 21, 3000, 64)])
def test_xent_backward(probe, T, V, D):
    st, got = probe("ufp4_linear_xent_bwd", HID, D, W, D, TG, T, V, D, 5 * P, 6 * P, 0, 7 * P, D, 8 * P, D,
                    WS, 1 << 62, 0)
    assert st == U.UFP4_OK
    assert ("k_zero_rows" if T == 0 else "k_slab_sum") in got[-1][0]


def test_xent_refuses_what_no_launch_takes():
    lib = U.lib_handle()
    for T, D in ((1 << 21, (1 << 17) + 8), ((1 << 18) + 1, 1 << 20)):
        assert lib.ufp4_linear_xent_fwd(HID, D, W, D, TG, T, 300, D, 5 * P, 6 * P, WS, 1 << 62,
                                        None) == U.UFP4_ERR_UNSUPPORTED
        assert lib.ufp4_linear_xent_bwd(HID, D, W, D, TG, T, 300, D, 5 * P, 6 * P, None, 7 * P, D, 8 * P, D,
                                        WS, 1 << 62, None) == U.UFP4_ERR_UNSUPPORTED
        assert U.ufp4_linear_xent_workspace_bytes(T, 300, D) == 0


def test_xent_forward_slices_write_their_own_tokens(probe):
    """A slice's statistics, target logits and targets start at its first token;
    the statistics' rows keep the pitch of all tokens."""
    T, V, D, part, part_ld, zt, targets = 1 << 21, 1 << 19, 8, 10, 11, 12, 13
    st, got = xent_fwd(probe, T, V, D, words="k_prod")
    assert st == U.UFP4_OK and len(got) > 3
    rows = V // 256 * 2
    at = 0
    for _, _, w in got[:-1]:
        assert w[part] == WS + 8 * at and w[part_ld] == T
        assert w[zt] == WS + 8 * rows * T + 4 * at and w[targets] == TG + 8 * at
        at += w[N_]
