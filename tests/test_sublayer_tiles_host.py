"""Which tiles the products take at the sizes that tests/test_gpu_gated_block_tiles.py
and tests/test_gpu_orthogonalize_tiles.py check (no GPU: the sources' own choice,
in a host build of them without the kernels)."""
import ctypes
import subprocess

import pytest

from param_collectives_amd import build
from tests.test_gpu_gated_block_tiles import SIZES
from tests.test_gpu_orthogonalize_tiles import SIZES as LISTS

PRINT = r"""
#include <cstdio>
void print(const char* name, const tide::Tiling& t) {
  std::printf(" %s %d %u %u %u %u", name, int(t.side), t.cut.tiles, t.cut.full, t.cut.splits, t.cut.items);
}
"""
MAIN = {"gated_block.hip": r"""
namespace tide {
bool rows_aligned(const void*, int64_t ld, int64_t cols) { return ld % 8 == 0 && cols % 8 == 0; }
int launch_align_rows(const void*, int64_t, int64_t, int64_t, void*, int64_t, void*, int64_t) { return 0; }
}
int main() {
  long long tokens, hidden, ffn;
  while (std::scanf("%lld %lld %lld", &tokens, &hidden, &ffn) == 3) {
    tide::GatedCall c{};
    c.tokens = tokens;
    c.hidden = c.x_ld = c.gate_ld = c.up_ld = hidden;
    c.ffn = ffn;
    c.grad = true;
    const Layout L = layout_of(c);
    std::printf("copies %d %d %lld", int(L.copy_x), int(L.copy_w), (long long)L.depth);
    print("forward", L.fwd);
    print("dx", L.dx);
    print("dw", L.dw);
    std::printf("\n");
  }
}
""", "orthogonalize.hip": r"""
int main() {
  long long count, rows, cols;
  while (std::scanf("%lld %lld %lld", &count, &rows, &cols) == 3) {
    tide::OrthogonalCall c{};
    c.count = int32_t(count);
    c.rows = rows;
    c.cols = cols;
    c.steps = 5;
    const Layout L = layout_of(c);
    const long long pieces = (count + L.piece - 1) / L.piece, last = count - (pieces - 1) * L.piece;
    for (long long n : {(long long)L.piece, last}) {
      const Tilings t = tilings_of(c, L, n);
      std::printf("pieces %lld %lld %lld %lld", pieces, n, (long long)L.partial_bytes, (long long)L.bytes);
      print("gram", t.gram);
      print("square", t.square);
      print("update", t.update);
      std::printf("\n");
    }
  }
}
"""}


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    """The lines that a source's choice prints for lines of sizes."""

    def of(source):
        at = tmp_path_factory.mktemp("tiles")
        (at / "main.hip").write_text(f'#include "{source}"\n{PRINT}{MAIN[source]}')
        (at / "none.c").write_text("const char __hip_fatbin[64] = {0};\n")  # in the place of the kernels' code
        subprocess.run([build.hipcc(), *build.FLAGS, "-Wno-unused-function", "-O1", "-fuse-cuid=none", "--offload-host-only", "-c",
                        str(at / "main.hip"), "-o", str(at / "main.o")], check=True, capture_output=True)
        subprocess.run(["gcc", "-fPIC", "-c", str(at / "none.c"), "-o", str(at / "none.o")], check=True)
        subprocess.run([build.hipcc(), "-no-hip-rt", str(at / "main.o"), str(at / "none.o"), "-o", str(at / "main"),
                        "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True)
        return lambda lines: subprocess.run([str(at / "main")], input="\n".join(lines), text=True, check=True,
                                            stdout=subprocess.PIPE).stdout.splitlines()

    return of


def products(line):
    """(words before the products, {product: (side, tiles, whole ones, splits, items)})."""
    words = line.split()
    at = [i for i, w in enumerate(words) if w.isalpha()]
    return words[:at[1]], {words[i]: tuple(map(int, words[i + 1:i + 6])) for i in at[1:]}


def test_the_blocks_products(program):
    lines = program("gated_block.hip")([" ".join(map(str, s)) for s in SIZES])
    one, copied, ragged = (products(line) for line in lines)
    # one round of whole tiles
    assert one[1]["forward"][0] == 256 and one[1]["forward"][3] == 1 and one[1]["forward"][4] <= 256
    # copies, filled up to whole steps; a split dx; dW by more tiles than there are places for
    assert copied[0] == ["copies", "1", "1", "4128"]
    assert copied[1]["forward"][0] == copied[1]["dx"][0] == copied[1]["dw"][0] == 256
    assert copied[1]["dx"][2:4] == (0, 7) and copied[1]["dw"][4] > 256 and copied[1]["dw"][3] == 1
    # of each product whole tiles and split ones, from a queue (dx's all split)
    for name in ("forward", "dx", "dw"):
        side, tiles, full, splits, items = ragged[1][name]
        assert side == 256 and splits > 1 and full < tiles
        assert name == "dx" or (full > 0 and items > 256)


def test_the_lists_products(program):
    lines = [products(line) for line in program("orthogonalize.hip")([" ".join(map(str, s)) for s in LISTS])]
    found = dict(zip(LISTS, zip(lines[::2], lines[1::2])))

    def of(size, name):
        return found[size][0][1][name]

    for size in LISTS[:2]:  # one round of whole tiles
        for name in ("gram", "square"):
            side, tiles, full, splits, items = of(size, name)
            assert side == 256 and splits == 1 and items <= 256
    for size in LISTS[2:4]:  # whole ones and split ones, from a queue
        for name in ("gram", "square", "update"):
            side, tiles, full, splits, items = of(size, name)
            assert side == 256 and splits > 1 and 0 < full < tiles and items > 256
    for size in LISTS[4:6]:
        side, tiles, full, splits, items = of(size, "update")
        assert side == 256 and splits > 1 and items > 256 and of(size, "gram")[0] == 128
    for size in LISTS[6:8]:
        assert of(size, "update")[0] == 256 and of(size, "update")[3] == 1 and of(size, "update")[4] > 256
    for size in LISTS[8:]:
        (words, first), (last_words, last) = found[size]
        assert int(words[1]) == 2 and int(words[2]) > int(last_words[2]) > 1
        assert all(first[n][0] != last[n][0] for n in ("gram", "square", "update"))
    # every orientation of each of these
    assert all(a[1] > a[2] and b[1] <= b[2] for a, b in ((LISTS[0], LISTS[1]), (LISTS[3], LISTS[2]), (LISTS[5], LISTS[4]),
                                                         (LISTS[7], LISTS[6]), (LISTS[8], LISTS[9])))


def test_workspaces_of_lists(program):
    """The matrices of a piece take 384 MiB at most, but one is always taken; the
    partial sums of three rounds of 256 tiles come to it, the queues and the norms."""
    from param_collectives_amd import tide

    sizes = [*LISTS, (128, 768, 2048), (128, 2048, 768), (4, 4096, 8200), (5000, 8, 8), (64, 2048, 2048), (300, 1000, 40)]
    lines = [products(line) for line in program("orthogonalize.hip")([" ".join(map(str, s)) for s in sizes])]
    for (count, rows, cols), (words, _) in zip(sizes, lines[::2]):
        piece, partial, need = map(int, words[2:5])
        got = ctypes.c_int64()
        assert tide.lib.tide_orthogonalize_workspace(count, rows, cols, 5, ctypes.byref(got)) == 0 and got.value == need
        assert partial <= 3 * 256 * 256 * 256 * 4
        small = min(rows, cols)
        # rows filled up to 32, columns to 64
        each = 3 * 2 * (-(-rows // 32) * 32) * (-(-cols // 64) * 64) + 2 * 2 * small * (-(-small // 64) * 64)
        assert piece == 1 or piece * each <= 3 << 27
        assert piece * each + partial < need < piece * each + partial + (1 << 20)
