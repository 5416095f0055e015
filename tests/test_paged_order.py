"""What no run of the paged attention can show, read from its source (no GPU)."""
import ctypes
import re
import subprocess

import pytest

from tests.test_la_order import source, statements


def test_a_wait_on_several_barriers_orders_memory_for_the_whole_warp():
    """Each of the barriers is seen by one lane, and another lane issues the products on what has
    arrived: a vote joins them, which orders no memory, so a barrier of the warp has to stand
    behind it."""
    code = source("kda_paged_tc.cuh")
    start = code.index("bool wait_warp(uint32_t bar0")
    body = statements(code[start:])[0]
    wins = re.findall(r"__all_sync\([^;{]*\)\)\s*(\{[^}]*\}|[^;{}]*;)", body)
    assert len(wins) == 1
    assert [x.strip("{} \n") for x in statements(wins[0].strip("{}\n "))[:2]] == ["__syncwarp();", "return true;"]


@pytest.fixture(scope="module")
def pieces(tmp_path_factory):
    """How the single-token kernel cuts an item's tiles into pieces, compiled for the host."""
    code = source("paged_decode_tc.cu")
    body = code[code.index("__device__ __forceinline__ int pieces("):code.index("template <int D, int NR, bool E4M3> struct Map")]
    most = re.search(r"constexpr int kTiles = (\d+);", code).group(1)
    where = tmp_path_factory.mktemp("pieces")
    (where / "pieces.cpp").write_text(
        "#include <algorithm>\nusing std::min;\n#define __device__\n#define __forceinline__\n"
        f"constexpr int kTiles = {most};\n{body}\n"
        'extern "C" int count_of(int tiles) { return pieces(tiles); }\n'
        'extern "C" int begin_of(int tiles, int u) { return piece_at(tiles, pieces(tiles), u); }\n')
    subprocess.run(["g++", "-O1", "-fwrapv", "-shared", "-fPIC", "-o", "pieces.so", "pieces.cpp"], cwd=where, check=True)
    lib = ctypes.CDLL(str(where / "pieces.so"))
    return lib.count_of, lib.begin_of, int(most)


@pytest.mark.parametrize("tiles", [1, 2, 4, 5, 7, 8, 9, 1000, 92680, 92681, 92682, 92683, 110377, (1 << 24) - 1, 1 << 24])
def test_pieces_of_any_length(pieces, tiles):
    """A context of up to 2^31 tokens has 2^24 tiles of 128 keys, all of which may be one CTA's: every
    piece begins where the one before ends and has 1 to kTiles tiles."""
    count_of, begin_of, most = pieces
    count = count_of(tiles)
    assert count == -(-tiles // most)
    some = range(count) if count < 30000 else [*range(8), *range(23168, 23176), *range(count // 2, count // 2 + 8),
                                               *range(count - 8, count)]
    for u in some:
        begin, end = begin_of(tiles, u), begin_of(tiles, u + 1)
        assert 0 <= begin < end <= begin + most and end <= tiles, u
    assert begin_of(tiles, 0) == 0 and begin_of(tiles, count) == tiles


def test_a_call_that_gives_up_leaves_nothing_to_be_joined():
    """The exit for shared memory that is not aligned (which no launch of today takes): the join reads the row of
    cuts, which is the workspace's old content unless the exit writes it."""
    code = source("paged_decode_tc.cu")
    start = code.index("if (base & 1023u)")
    leave = statements(code[start:])[0]
    assert "return;" in leave
    assert re.search(r"p\.cuts\[[^;]*\] = Cut\{0, 0, 0, 0, 0\};", leave[:leave.index("return;")])
