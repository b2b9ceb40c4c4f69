"""How the feed-forward products cut their reductions, on the host: the
functions that every warp of the kernel counts by, replayed warp by warp."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    out = str(tmp_path_factory.mktemp("replay") / "replay.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "mot_dit_b200", "csrc"),
                    os.path.join(ROOT, "tests", "c_abi", "reduction_replay.cpp"), "-o", out], check=True)
    return C.CDLL(out)


@pytest.mark.parametrize("subs", [1, 2])
@pytest.mark.parametrize("chain", [0, 12, 14])
def test_segments_of_any_part(replay, subs, chain):
    """Parts of every length, with and without a seam between operand pairs in them."""
    for n in range(1, 200):
        for seam in [0, n, *range(1, n, 1 if n < 60 else 7)]:
            lo = 3
            assert replay.replay_part(lo, lo + n, lo + seam, subs, chain, 0) == 0, (n, seam)
            for nseg in (1, 3, 6) if subs == 1 else ():  # fp32 operands: rounds of segments
                assert replay.replay_part(lo, lo + n, lo + seam, subs, chain, nseg) == 0, (n, seam)


@pytest.mark.parametrize("sides", [1, 2])
@pytest.mark.parametrize("f32", [0, 1])
def test_segments_of_every_width(replay, f32, sides):
    """The MMA warp closes as many accumulator segments as the epilogue waits for, at every width of a layer (with two
    operand pairs, a piece that crosses the seam after an odd number of k-blocks had one segment fewer)."""
    rows = (1, 16, 64, 256, 640, 2048, 8448)
    for N in range(64, 32769, 64):  # (the counts go by k-blocks of 64)
        for K in (64, 256, 512, 1024, 1536, 2048, 4096):
            for M in rows:
                assert replay.replay_backward(f32, M, N, K, sides) == 0, (M, N, K)


@pytest.mark.parametrize("M,F,K", [(256, 8192, 1024), (16, 8192, 1536), (128, 8192, 1536), (64, 8192, 2048), (2048, 8192, 256)])
def test_widths_that_a_seam_cuts(replay, M, F, K):
    """Shapes whose input gradient is cut into three pieces, the middle one across the seam."""
    assert replay.pieces_dx(0, M, F, K, 2) == 3
    kb0 = F // 64
    assert replay.replay_part(2 * kb0 // 3, 4 * kb0 // 3, kb0, 2, 14, 0) == 0


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("b_mn", [0, 1])
def test_tile_widths(replay, gated, b_mn):
    """fp32 tiles are as wide as one of the two loaders (a linear layer of up to 32 or of 65 to 96 columns had tiles of 32
    or 96, which neither brings in); the others are whole boxes."""
    for N in range(1, 400):
        need = 2 * ((N + 31) // 32 * 32) if gated else N
        for bn in (64, 128):
            c = replay.columns(bn, N, gated, b_mn, 0, 1)
            assert c in (64, 128) and c <= bn and (c == bn or c >= need), (N, bn, c)
        for bn in range(64, 257, 32):
            c = replay.columns(bn, N, gated, b_mn, 0, 0)
            assert c <= bn and c % (64 if (gated or b_mn) and bn % 64 == 0 else 32) == 0 and (c == bn or need <= c < need + 64)
        for bn in (128, 192, 256):
            c = replay.columns(bn, N, gated, b_mn, 1, 0)
            assert c <= bn and c % 64 == 0 and (c == bn or need <= c < need + 128)


def test_fp32_chains_stay_short(replay):
    """A reduction of any length: no accumulator of an fp32 product sums more than 12 k-blocks (there were seven segments
    at most, as long as it took)."""
    for n in [*range(1, 400), 1024, 2048, 4000]:
        assert replay.longest_chain(n, 1, 12) <= 12, n
        assert replay.longest_chain(n, 2, 14) <= 14, n


@pytest.mark.parametrize("stream,rest", [(4, 2), (2, 2), (4, 4)])
def test_norm_blocks_fit_as_planned(replay, stream, rest):
    """The chunks of the backward norm count on as many blocks an SM as its shared memory holds (at 32, 64, 128, 256 and
    1792 columns of fp32 one ran where two were planned)."""
    stages, planned = C.c_int(), C.c_int()
    for D in range(1, 8193):
        need = replay.grad_block(D, stream, rest, C.byref(stages), C.byref(planned))
        assert stages.value >= 1 and need * planned.value <= 227 * 1024, (D, need, planned.value)
