"""Which tiles the block's products take at the sizes that
tests/test_gpu_gated_block_tiles.py checks (no GPU: the source's own choice, in a
host build of it without the kernels)."""
import subprocess

import pytest

from param_collectives_amd import build
from tests.test_gpu_gated_block_tiles import SIZES

MAIN = {"gated_block.hip": r"""
namespace tide {
bool rows_aligned(const void*, int64_t ld, int64_t cols) { return ld % 8 == 0 && cols % 8 == 0; }
int launch_align_rows(const void*, int64_t, int64_t, int64_t, void*, int64_t, void*, int64_t) { return 0; }
}
void print(const char* name, const tide::Tiling& t) {
  std::printf(" %s %d %u %u %u %u", name, int(t.side), t.cut.tiles, t.cut.full, t.cut.splits, t.cut.items);
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
"""}


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    """The lines that a source's choice prints for lines of sizes."""

    def of(source):
        at = tmp_path_factory.mktemp("tiles")
        (at / "main.hip").write_text(f'#include "{source}"\n#include <cstdio>\n{MAIN[source]}')
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
